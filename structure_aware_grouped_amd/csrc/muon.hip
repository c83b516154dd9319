// Orthogonalisation of whole matrices by Newton-Schulz products, and the Muon
// step built on it, on gfx950: kernels and the rs_orthogonalize /
// rs_muon_step / rs_muon_workspace entry points ("veScale-FSDP: flexible,
// structure-aware sharding at 10K-GPU scale", feynmanwiki walkthrough, Muon
// paragraphs: a rank that holds a whole matrix runs Newton-Schulz on it).
//
// Mathematics, for a matrix G (X is G or its transpose, m x n with m <= n):
//   X <- G / (|G|_F + eps);  `steps` times:  X <- (a I + b A + c A^2) X,
//   A = X X^T.
// Every product has the form  C[i, j] = sum_k P[i, k] Q[j, k]  with k
// contiguous in both operands: A from X and X; A^2 from A and A (symmetric);
// the polynomial times X from the symmetric polynomial and X^T, which is kept
// beside X. A and A^2 are symmetric, so only tiles on and below the diagonal
// are computed and each is stored twice.
//
// Number formats. Products run on fp16 operands with fp32 sums
// (v_mfma_f32_32x32x16_f16): at the same rate as bf16, fp16 rounds 8 times
// finer, and every operand here has a known size, so fp16's range is no
// limit: X is stored times 2^ex (about sqrt(n)), A and the polynomial times
// 2^10. Three things that fp16 alone would spoil are kept apart:
//   - X as a high and a low fp16 part. A gradient with few strong directions
//     has its weak ones below the rounding error of the strong ones, and the
//     steps raise them. With the polynomial as d_i on the diagonal (fp32)
//     plus the rest (fp16), d_i acts on both parts and only the rest is
//     multiplied with the high part alone. While a row of X is short (A_ii at
//     most 1/2: early steps) d_i = a, so the rest spans the strong directions
//     only and drops nothing from the weak ones; later d_i is the whole
//     diagonal, so the rest is small where A is near the identity.
//   - the diagonal of A in fp32, zeros in its place in the fp16 operand.
// A matrix of few rows has few singular values, so its error is that of the
// worst of them, and the published polynomial's slope reaches 1.6: for
// m <= kMatTwoPart, and for every matrix of a plan loaded with muon_parts = 2,
// all operands have a high and a low part, and a product is
// high * low + low * high + high * high.
// On matrices of 100 to 2048 rows with one part, with spectra flat, falling by
// 10^4 or of a few directions 100 times above the others, the relative error
// of the result against 64 bits is 2e-4 to 1.2e-3 (computed with the same
// roundings on the CPU); plain fp16 operands give 1e-3 to 4e-2, bf16 ones 1e-2
// and more. Two parts for every matrix give 4e-7 to 1.2e-6 on the card (one:
// 2.3e-4 to 9.6e-4), 1.4e-5 where most directions are 100 times weaker than a
// few (fp32 products give 2.8e-5 there), at 1.4 (100 x 110) to 2.9
// (4096 x 14336: 4.0 -> 11.8 ms) times the time, so one is the default: its
// error is below the bf16 rounding of rs_orthogonalize's result (where it moves
// 16 to 22% of the values to their bf16 neighbour), and in rs_muon_step it comes
// times the rate.
//
// What bounds it. The products: with 256-wide tiles the matrix cores are busy
// 61 to 73% of the time for 8192 x 28672, at the 1.6 to 1.7 GHz that the card
// holds under them (polynomial times X 3.41 ms, 1128 TFLOP/s, X X^T 1204; a
// library fp16 product of that size reaches 1373 to 1427), and 42 to 58% at 1.8
// GHz for the Llama-3-8B layer. Small matrices: the latency of about 17
// launches. The passes around the products move bytes: momentum and norm 5.7
// TB/s, the split into operands 4.8 TB/s on that layer's 218 M elements, 8% of
// its 14.4 ms.
#include "host_common.h"

namespace rs {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr float kOpScale = 1024.0f;          // stored A and polynomial: value * 2^10
constexpr float kLowScale = 2048.0f;         // stored low part of X: (x - high) * 2^11

// What a call does to each matrix beside the products.
struct MuonK {
  float a, b, c;       // polynomial of this step
  float mu;            // momentum decay
  float lr, decay;     // decay = 1 - lr * weight_decay
  int32_t nesterov, scale_mode;
};

__device__ __forceinline__ float load_elem(const void* p, int64_t i, bool bf16) {
  return bf16 ? In<true>::elem(p, i) : In<false>::elem(p, i);
}

// ------------------------------------------------------------------ momentum and norm

// One chunk of one matrix: m <- mu m + g (fp32, in place) where there is a
// momentum, and the chunk's sum of squares of the matrix to orthogonalise
// (g, m, or g + mu m). Squares and sums are fp64: an fp32 square would
// overflow from 1e19 and vanish below 1e-23.
template <bool BF16, bool MUON>
__global__ __launch_bounds__(kThreads) void mat_norm_kernel(const MuonMat* __restrict__ mats,
                                                            const MatChunk* __restrict__ jobs, const void* grad,
                                                            float* mom, char* work, MuonK k) {
  __shared__ double red[kThreads / kWave];
  const MatChunk job = jobs[blockIdx.x];
  const MuonMat& q = mats[job.mat];
  const int64_t n = static_cast<int64_t>(q.rows) * q.cols, off = static_cast<int64_t>(job.chunk) * kMatChunk;
  const int64_t base = q.start + off;
  const int len = static_cast<int>(n - off < kMatChunk ? n - off : kMatChunk);
  double sum = 0.0;
  auto one = [&](float g, float& m) {
    if constexpr (MUON) {
      m = __fadd_rn(__fmul_rn(k.mu, m), g);
      g = k.nesterov ? __fadd_rn(g, __fmul_rn(k.mu, m)) : m;
    }
    sum += static_cast<double>(g) * static_cast<double>(g);
  };
  const int nv = len / 8;   // base is a multiple of 16 elements
  for (int v = threadIdx.x; v < nv; v += kThreads) {
    float x[8], m[8] = {};
    if constexpr (BF16) {
      In<true>::widen(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(grad) + base + v * 8), x);
    } else {
      const f32x4* gp = reinterpret_cast<const f32x4*>(static_cast<const float*>(grad) + base + v * 8);
      const f32x4 g0 = gp[0], g1 = gp[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) { x[e] = g0[e]; x[4 + e] = g1[e]; }
    }
    f32x4* mp = reinterpret_cast<f32x4*>(mom + base + v * 8);
    if constexpr (MUON) {
      const f32x4 m0 = mp[0], m1 = mp[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) { m[e] = m0[e]; m[4 + e] = m1[e]; }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) one(x[e], m[e]);
    if constexpr (MUON) {
      mp[0] = f32x4{m[0], m[1], m[2], m[3]};
      mp[1] = f32x4{m[4], m[5], m[6], m[7]};
    }
  }
  for (int e = nv * 8 + threadIdx.x; e < len; e += kThreads) {
    float m = 0.0f;
    if constexpr (MUON) m = mom[base + e];
    one(load_elem(grad, base + e, BF16), m);
    if constexpr (MUON) mom[base + e] = m;
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / kWave; ++w) sum += red[w];
    reinterpret_cast<double*>(work + q.part)[job.chunk] = sum;
  }
}

// 2^ex / (norm + eps) of a matrix, by one workgroup; the partial sums are
// added in a fixed order.
__device__ __forceinline__ double mat_scale(const MuonMat& q, const char* work, double eps, double* red) {
  const double* part = reinterpret_cast<const double*>(work + q.part);
  double sum = 0.0;
  for (int i = threadIdx.x; i < q.n_part; i += kThreads) sum += part[i];
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < kThreads / kWave; ++w) sum += red[w];
  return static_cast<double>(1 << q.ex) / (sqrt(sum) + eps);
}

// The same for every matrix ahead of the split, where adding up the sums in
// every workgroup of the split would cost more than a launch.
__global__ __launch_bounds__(kThreads) void mat_scale_kernel(const MuonMat* __restrict__ mats, char* work, double eps) {
  __shared__ double red[kThreads / kWave];
  const MuonMat& q = mats[blockIdx.x];
  const double inv = mat_scale(q, work, eps, red);
  if (threadIdx.x == 0) *reinterpret_cast<double*>(work + q.inv) = inv;
}

// x as a high and a low fp16 part.
__device__ __forceinline__ void split(float x, _Float16& hi, _Float16& lo) {
  hi = static_cast<_Float16>(x);
  lo = static_cast<_Float16>((x - static_cast<float>(hi)) * kLowScale);
}

// One 64 x 64 tile of X from the gradient (and momentum): scaled, split, and
// written as X's high and low parts and the transposed high part (with two
// parts the low one too), zeros in the padding of the contraction dimensions.
template <bool BF16, bool MUON>
__global__ __launch_bounds__(kThreads) void mat_spread_kernel(const MuonMat* __restrict__ mats,
                                                              const MatJob* __restrict__ jobs, const void* grad,
                                                              const float* mom, char* work, MuonK k, bool own_scale,
                                                              double eps) {
  constexpr int T = kMatSpread;
  __shared__ float tile[T][T + 1];   // [row of X][column of X]
  __shared__ double red[kThreads / kWave];
  const MatJob job = jobs[blockIdx.x];
  const MuonMat& q = mats[job.mat];
  const double inv = own_scale ? mat_scale(q, work, eps, red) : *reinterpret_cast<const double*>(work + q.inv);
  const int i0 = job.i * T, j0 = job.j * T;
  // the matrix's own rows r0.. and columns c0.. ; element (r, c) is X's (r, c) or (c, r)
  const int r0 = q.tall ? j0 : i0, c0 = q.tall ? i0 : j0;
  auto put = [&](int r, int c, float g, float m) {
    if constexpr (MUON) g = k.nesterov ? __fadd_rn(g, __fmul_rn(k.mu, m)) : m;
    const float x = static_cast<float>(static_cast<double>(g) * inv);
    if (q.tall) tile[c][r] = x;
    else tile[r][c] = x;
  };
  if (q.cols % 4 == 0) {   // four neighbours per load, all of a thread's loads first
    constexpr int kIt = T * T / 4 / kThreads;
    const int c = threadIdx.x % (T / 4) * 4;
    f32x4 g[kIt], m[kIt];
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int r = threadIdx.x / (T / 4) + it * (kThreads / (T / 4));
      g[it] = m[it] = f32x4{};
      if (r0 + r < q.rows && c0 + c < q.cols) {
        const int64_t at = q.start + static_cast<int64_t>(r0 + r) * q.cols + c0 + c;
        if constexpr (BF16) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(grad) + at);
          g[it] = f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xffff0000u)};
        } else {
          g[it] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(grad) + at);
        }
        if constexpr (MUON) m[it] = *reinterpret_cast<const f32x4*>(mom + at);
      }
    }
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int r = threadIdx.x / (T / 4) + it * (kThreads / (T / 4));
      const bool in = r0 + r < q.rows && c0 + c < q.cols;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (in) put(r, c + t, g[it][t], m[it][t]);
        else if (q.tall) tile[c + t][r] = 0.0f;
        else tile[r][c + t] = 0.0f;
      }
    }
  } else {   // single elements; again a thread's loads first
    constexpr int kIt = T * T / kThreads;
    const int c = threadIdx.x % T;
    float g[kIt], m[kIt];
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int r = threadIdx.x / T + it * (kThreads / T);
      g[it] = m[it] = 0.0f;
      if (r0 + r < q.rows && c0 + c < q.cols) {
        const int64_t at = q.start + static_cast<int64_t>(r0 + r) * q.cols + c0 + c;
        g[it] = load_elem(grad, at, BF16);
        if constexpr (MUON) m[it] = mom[at];
      }
    }
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int r = threadIdx.x / T + it * (kThreads / T);
      if (r0 + r < q.rows && c0 + c < q.cols) put(r, c, g[it], m[it]);
      else if (q.tall) tile[c][r] = 0.0f;
      else tile[r][c] = 0.0f;
    }
  }
  __syncthreads();
  _Float16* xh = reinterpret_cast<_Float16*>(work + q.xh);
  _Float16* xl = reinterpret_cast<_Float16*>(work + q.xl);
  _Float16* xt0 = reinterpret_cast<_Float16*>(work + q.xt[0]);
  for (int e = threadIdx.x; e < T * T / 8; e += kThreads) {
    const int r = e / (T / 8), c = e % (T / 8) * 8;
    if (i0 + r < q.m) {   // row r of X, 8 columns
      h8 hi, lo;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        _Float16 h, l;
        split(tile[r][c + t], h, l);
        hi[t] = h;
        lo[t] = l;
      }
      const int64_t at = static_cast<int64_t>(i0 + r) * q.np + j0 + c;
      *reinterpret_cast<h8*>(xh + at) = hi;
      *reinterpret_cast<h8*>(xl + at) = lo;
    }
    if (j0 + r < q.n) {   // column r of X, 8 rows
      h8 hi, lo;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        _Float16 h, l;
        split(tile[c + t][r], h, l);
        hi[t] = h;
        lo[t] = l;
      }
      const int64_t at = static_cast<int64_t>(j0 + r) * q.mp + i0 + c;
      *reinterpret_cast<h8*>(xt0 + at) = hi;
      if (q.two_part) *reinterpret_cast<h8*>(reinterpret_cast<_Float16*>(work + q.xtl[0]) + at) = lo;
    }
  }
}

// ------------------------------------------------------------------ products

enum Product {
  P_GRAM,    // A = X X^T: off-diagonal part and diagonal
  P_POLY,    // a I + b A + c A^2: off-diagonal part and diagonal
  P_MUL,     // a product of two polynomials in A: off-diagonal part and diagonal
  P_APPLY,   // polynomial times X: the next X
  P_OUT,     // the same, last step: the result in bf16
  P_STEP     // the same, last step: the parameters' update
};

// The first two steps of a paired matrix as one. With P = a I + b A + c A^2
// the first one's polynomial, X X^T becomes P A P, so the second polynomial
// can be had without X:
//   A (P_GRAM), P (P_POLY), T = P A, A1 = T P (P_MUL), Q = a' I + b' A1 + c' A1^2
//   (P_POLY), S = Q P (P_MUL), X <- S X (P_APPLY).
// All of them are polynomials in A, so symmetric, and each product costs m^3;
// X X^T and S X, the long products, are needed once. The rounding of A reaches
// further than in a single step: it is raised by a^2, so this is done only for
// |a| <= kPairMaxA and for the first two steps, where the singular values are
// small (the same error as single steps; the third and fourth as one gave 2 to
// 5 times the error). 8192 x 28672: 29.2 -> 25.9 ms a step.
enum PairPart { kPairT = 0, kPairA1 = 1, kPairS = 2 };
constexpr float kPairMaxA = 4.0f;

// Where the operands and the result of one product of one matrix lie, in the
// workspace. pair: the second of two paired steps (P_POLY, P_APPLY), or which
// product (P_MUL).
struct Where {
  int64_t p, q, out, dp, dq, dout;   // offdiagonal parts and diagonals
  int turn;                          // which transposed X is read
};

template <Product WHAT>
__device__ __forceinline__ Where where(const MuonMat& m, int turn, int pair) {
  if constexpr (WHAT == P_GRAM) return {m.xh, m.xh, m.a, 0, 0, m.da, 0};
  if constexpr (WHAT == P_POLY) {
    return pair && m.paired ? Where{m.a, m.a, m.c, m.da2, m.da2, m.dc, 0} : Where{m.a, m.a, m.b, m.da, m.da, m.db, 0};
  }
  if constexpr (WHAT == P_MUL) {
    return pair == kPairT    ? Where{m.b, m.a, m.t, m.db, m.da, m.dt, 0}
           : pair == kPairA1 ? Where{m.t, m.b, m.a, m.dt, m.db, m.da2, 0}
                             : Where{m.c, m.b, m.t, m.dc, m.db, m.dt, 0};
  }
  // paired matrices have changed X once less
  const int from = m.paired && turn > 0 && pair >= 0 ? (turn - 1) & 1 : turn & 1;
  const bool s = pair == 1 && m.paired;
  return {s ? m.t : m.b, m.xt[from], m.xt[from ^ 1], s ? m.dt : m.db, 0, 0, from};
}

// C = P Q^T on one BM x BM output tile by a 2 x WC grid of waves, each with
// NI x NJ accumulators of 32 x 32. Operands go straight from memory to LDS,
// kMatK wide, in kStages stages: while one is multiplied the others are on
// their way. In LDS a row is 128 bytes, eight 16-byte pieces, piece c of row
// r at place c ^ (r / 2 % 8): two rows fill the 64 banks once, and any 16
// neighbouring rows of a fragment spread over all of them; the loads permute
// the pieces within each row's 128-byte line in memory. The fragment of the
// next 16 columns is read while the current one is multiplied; the stage turns
// over (wait, barrier, new loads) before the last multiplication of a stage.
//   256: 64 KiB a stage, one workgroup per CU; what large products take. 128
// and 64: two workgroups per CU, for products of few tiles; 64 keeps three
// stages on their way, since few workgroups wait for memory. Whole calls, 64 /
// 128 / 256 wide: 1024 x 4096 248 / 339 / 569 us, 4096 x 4096 2.27 / 1.60 /
// 1.75 ms, 4096 x 14336 5.84 / 4.00 / 4.01 ms (3.85 with the rule: 128 for the
// m x m products, 256 for the m x n ones).
template <int BM>
struct Tile {
  static constexpr int kNT = BM == 256 ? 512 : 256;
  static constexpr int kWaves = kNT / kWave;
  static constexpr int WC = kWaves / 2;          // wave columns
  static constexpr int NI = BM / 64;             // 32-row blocks per wave
  static constexpr int NJ = BM / (32 * WC);      // 32-column blocks per wave
  static constexpr int kStages = BM == 64 ? 4 : 2;
  static constexpr int kStage = 2 * BM * kMatK * 2;   // bytes of both operands
  static constexpr int kLds = kStages * kStage;
  static constexpr int kLoads = kStage / 1024 / kWaves;   // 1 KiB loads per wave and stage
  static constexpr int IB = NI < 2 ? NI : 2;     // 32-row blocks of a wave that are stored in one pass
  static constexpr int kPasses = NI / IB;
};

// Waits for all but VM of the wave's loads (and LDS reads, with LGKM). The
// builtin, unlike assembly text, tells the compiler what has arrived.
template <int VM, bool LGKM>
__device__ __forceinline__ void wait() {
  static_assert(VM < 64, "a six-bit counter");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (VM >> 4) << 14 | 0x70 | (LGKM ? 0 : 0xf00));
}

// Workgroup barrier without a wait of its own; no memory access moves across.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The thread's number, as a value that the compiler cannot see through: what
// is computed from it is computed anew for each tile instead of being kept in
// registers through the multiplication, which needs all of them.
__device__ __forceinline__ int fresh_thread() {
  int t = static_cast<int>(threadIdx.x);
  asm volatile("" : "+v"(t));
  return t;
}

template <int BM>
struct Acc {
  f32x16 v[Tile<BM>::NI][Tile<BM>::NJ];
};

template <int BM>
struct Multiply {
__device__ static __forceinline__ void run(const _Float16* P, const _Float16* Q, int ld, int p0, int p_rows, int q0,
                                         int q_rows, int k0, int k1, char* lds, Acc<BM>& c) {
  using T = Tile<BM>;
  const int ksteps = k1 - k0;
  const int tid = fresh_thread();
  const int lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wr = wave / T::WC, wc = wave % T::WC;
  // rows past an operand's end repeat its last row: their results are not stored
  const int64_t row_bytes = static_cast<int64_t>(ld) * 2;
  const int pr = min(p_rows - p0, BM), qr = min(q_rows - q0, BM);
  const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(reinterpret_cast<const char*>(P) + p0 * row_bytes), 0, static_cast<int>(pr * row_bytes),
      kRawBufferWord3);
  const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(reinterpret_cast<const char*>(Q) + q0 * row_bytes), 0, static_cast<int>(qr * row_bytes),
      kRawBufferWord3);
  constexpr int kHalf = T::kLoads / 2;   // the first half of the loads fetch P, the others Q
  int off[T::kLoads];
#pragma unroll
  for (int t = 0; t < T::kLoads; ++t) {
    const int seg = (t % kHalf) * T::kWaves + wave;
    const int row = min(seg * 8 + lane / 8, (t < kHalf ? pr : qr) - 1);
    off[t] = static_cast<int>(row * row_bytes) + ((lane % 8) ^ ((seg * 8 + lane / 8) / 2 % 8)) * 16;
  }
  // LDS: P's stages, then Q's, so that a stage and a block are immediate
  // offsets of a fragment read
  constexpr int kHalfStage = T::kStage / 2;
  auto load = [&](int s, int stage) {
    const int k = (k0 + s) * static_cast<int>(kMatK) * 2;
#pragma unroll
    for (int t = 0; t < T::kLoads; ++t) {
      lds_char* dst = (lds_char*)lds + (t < kHalf ? 0 : T::kStages * kHalfStage) + stage * kHalfStage + wave * 1024 +
                      (t % kHalf) * T::kWaves * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(t < kHalf ? rp : rq, dst, 16, off[t], k, 0, 0);
    }
  };
  // fragment addresses: row lane % 32 of a block, columns kk*16 + lane/32*8 ..+7
  const int frow = lane % 32;
  const char *fp[4], *fq[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const int at = frow * 128 + (((kk * 2 + lane / 32) ^ (frow / 2 % 8)) * 16);
    fp[kk] = lds + at + wr * T::NI * 32 * 128;
    fq[kk] = lds + at + T::kStages * kHalfStage + wc * T::NJ * 32 * 128;
  }
  h8 fa[2][T::NI], fb[2][T::NJ];
  auto fetch = [&](int stage, int kk, int to) {
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) fb[to][j] = *reinterpret_cast<const h8*>(fq[kk] + stage * kHalfStage + j * 4096);
#pragma unroll
    for (int i = 0; i < T::NI; ++i) fa[to][i] = *reinterpret_cast<const h8*>(fp[kk] + stage * kHalfStage + i * 4096);
  };
  auto mma = [&](int from) {
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
      for (int j = 0; j < T::NJ; ++j)
        c.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[from][i], fb[from][j], c.v[i][j], 0, 0, 0);
  };
  // one fragment read between multiplications, so that none of them waits
  constexpr int kReads = T::NI + T::NJ, kMuls = T::NI * T::NJ, kPairs = kReads < kMuls ? kReads : kMuls;
  auto interleave = [&]() {
    if constexpr (kReads > kPairs) __builtin_amdgcn_sched_group_barrier(0x100, kReads - kPairs, 0);   // LDS reads
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one multiplication
    }
    if constexpr (kMuls > kPairs) __builtin_amdgcn_sched_group_barrier(0x008, kMuls - kPairs, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // One stage: three sixteen-column multiplications, each while the next
  // fragment is read; then, with every wave done reading this stage and the
  // next stage arrived (full: later ones may still be on their way), the loads
  // into this stage and the next stage's first fragment, under the fourth.
  constexpr int S = T::kStages;
  auto step = [&](int s, int stage, int next, bool full, bool more_loads, bool more) {
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) {
      fetch(stage, kk + 1, (kk + 1) & 1);
      mma(kk & 1);
      interleave();
    }
    if (full) wait<(S - 2) * T::kLoads, true>();
    else wait<0, true>();
    barrier();
    if (more) fetch(next, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    if (more_loads) load(s + S, stage);
    __builtin_amdgcn_sched_barrier(0);
    mma(1);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < ksteps) load(s, s);
  if (ksteps >= S) wait<(S - 1) * T::kLoads, false>();
  else wait<0, false>();
  barrier();
  fetch(0, 0, 0);
  int s = 0;
  for (; s + 2 * S - 1 < ksteps; s += S) {
#pragma unroll
    for (int u = 0; u < S; ++u) step(s + u, u, (u + 1) % S, true, true, true);
  }
  for (; s < ksteps; ++s) step(s, s % S, (s + 1) % S, s + S <= ksteps, s + S < ksteps, s + 1 < ksteps);
}
};

// sqrt(max(1, rows / cols)), 0.2 sqrt(max(rows, cols)) or 1.
__device__ __forceinline__ float update_scale(int mode, int rows, int cols) {
  if (mode == RS_MUON_SCALE_SPECTRAL) return rows > cols ? sqrtf(static_cast<float>(rows) / cols) : 1.0f;
  if (mode == RS_MUON_SCALE_RMS) return 0.2f * sqrtf(static_cast<float>(max(rows, cols)));
  return 1.0f;
}

// The sums of one part of a cut tile. Slab element order is that of the
// registers: 16 bytes per thread.
template <int BM>
struct Slab {
using T = Tile<BM>;
static constexpr int kBytes = BM * BM * 4;

__device__ static __forceinline__ __amdgpu_buffer_rsrc_t at(char* slabs, int slab) {
  return __builtin_amdgcn_make_buffer_rsrc(slabs + static_cast<int64_t>(slab) * kBytes, 0, kBytes, kRawBufferWord3);
}

__device__ static __forceinline__ void store(const Acc<BM>& acc, char* slabs, int slab) {
  const int mine = fresh_thread() * 16;
  const __amdgpu_buffer_rsrc_t r = at(slabs, slab);
#pragma unroll
  for (int i = 0; i < T::NI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x4 x = {acc.v[i][j][4 * e], acc.v[i][j][4 * e + 1], acc.v[i][j][4 * e + 2], acc.v[i][j][4 * e + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, mine, ((i * T::NJ + j) * 4 + e) * T::kNT * 16, 0);
      }
}

// The sums over all parts of block row `strip` (32 rows of the tile), in the
// order of the parts, by WC waves.
__device__ static __forceinline__ void add(f32x16 (&v)[1][T::NJ], char* slabs, int slab, int parts, int strip) {
  const int mine = (strip / T::NI * T::WC * kWave + fresh_thread()) * 16;
  const int base = strip % T::NI * T::NJ * 4 * T::kNT * 16;
#pragma unroll
  for (int j = 0; j < T::NJ; ++j) v[0][j] = f32x16{};
#pragma unroll 2
  for (int p = 0; p < parts; ++p) {
    const __amdgpu_buffer_rsrc_t r = at(slabs, slab + p);
    f32x4 x[T::NJ][4];
#pragma unroll
    for (int j = 0; j < T::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[j][e] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, mine, base + (j * 4 + e) * T::kNT * 16, 0));
#pragma unroll
    for (int j = 0; j < T::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int t = 0; t < 4; ++t) v[0][j][4 * e + t] += x[j][e][t];
  }
}
};

// What is stored of some rows of one tile: in a product, of IB 32-row blocks of
// each of the NW = 2 wave rows (a pass); in a join, of one block (NW = IB = 1).
// The sums go through LDS: a row-wise phase
// computes the result and stores it along its rows, a column-wise phase stores
// its transpose. In LDS element (r, j) lies at r * BM + (j ^ 4 * (r / 8 % 16)):
// 16-byte pieces along a row stay whole, and the eight rows that a lane of the
// column-wise phase reads fall into banks of their own. Row r of these is the
// tile's row r / (32 IB) * 32 NI + base + r % (32 IB).
//   In the row-wise phase a thread has eight columns of kRows rows. What it
// reads of them from memory is fetched kAhead rows at a time, the first ones
// before the sums go to LDS: one row at a time the loads of a row waited for
// the stores of the one before (20 us for one 128-wide tile).
template <int BM, Product WHAT, int NW, int IB>
struct Store {
using T = Tile<BM>;
static constexpr int kNT = NW * T::WC * kWave;
static constexpr int kHeight = NW * IB * 32;
static constexpr int kBytes = kHeight * BM * 4;   // of LDS
static constexpr bool kSym = WHAT == P_GRAM || WHAT == P_POLY || WHAT == P_MUL;
static constexpr bool kLast = WHAT == P_OUT || WHAT == P_STEP;
static constexpr int kRows = kHeight * (BM / 8) / kNT, kRowStep = kNT / (BM / 8);
static constexpr int kAhead = WHAT == P_STEP || WHAT == P_MUL || (WHAT == P_POLY && BM == 256) || kRows < 4 ? 2 : 4;
static constexpr int kCols = BM * (kHeight / 8) / kNT, kColStep = kNT / (kHeight / 8);
static_assert(kRows % kAhead == 0 && kRows * kRowStep == kHeight && kCols * kColStep == BM, "whole rows and columns");

struct In8 {   // of one row: A (POLY) or X, high and low; both factors (MUL); parameters (STEP)
  h8 hi, lo;
  float d;
  f32x4 p[2];
};

// Rounded to bf16, or subtracted from the parameters; e elements from dst on
// lie inside the matrix, whole: 16-byte aligned and all eight inside.
__device__ static __forceinline__ void finish(void* out, int64_t at, const float (&v)[8], int e, bool whole, float f,
                                              float decay, const f32x4 (&p)[2]) {
  if constexpr (WHAT == P_OUT) {
    uint16_t* dst = static_cast<uint16_t*>(out) + at;
    uint32_t w[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) w[t] = bf16_rne(v[t] * f);
    if (whole) {
      *reinterpret_cast<u32x4*>(dst) = u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < e) dst[t] = static_cast<uint16_t>(w[t]);
    }
  } else {
    float* dst = static_cast<float*>(out) + at;
    if (whole) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 x;
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = __fsub_rn(__fmul_rn(p[h][t], decay), __fmul_rn(f, v[4 * h + t]));
        reinterpret_cast<f32x4*>(dst)[h] = x;
      }
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < e) dst[t] = __fsub_rn(__fmul_rn(dst[t], decay), __fmul_rn(f, v[t]));
    }
  }
}

// acc: the sums of each wave's IB block rows; base: the tile's row of row 0.
__device__ static __forceinline__ void run(const f32x16 (&acc)[IB][T::NJ], const ProductJob& job, const MuonMat& q,
                                           int base, char* work, char* lds, int turn, int pair, const MuonK& k,
                                           void* out) {
  const Where at_ = where<WHAT>(q, turn, pair);
  const int i0 = job.i * BM, j0 = job.j * BM;
  const int m = q.m, n = q.n, mp = q.mp, np = q.np;
  const bool two = q.two_part, tall = q.tall;
  const int jn = kSym ? m : n, jp = kSym ? mp : np;   // columns of this product, and padded
  const int tid = fresh_thread(), lane = tid % kWave, wave = tid / kWave;
  const int wr = wave / T::WC, wc = wave % T::WC;
  float* stage = reinterpret_cast<float*>(lds);
  const float ex = static_cast<float>(1 << q.ex);
  // factor of the stored X in the result
  const float f = WHAT == P_STEP ? k.lr * update_scale(k.scale_mode, q.rows, q.cols) / ex : 1.0f / ex;
  float* diag = reinterpret_cast<float*>(work + (WHAT == P_GRAM ? at_.dout : at_.dp));

  // row-wise: rows i0 + row(it), columns j .. j + 7
  const int r0 = tid / (BM / 8), c = tid % (BM / 8) * 8, j = j0 + c;
  auto tile_row = [&](int r) { return i0 + r / (IB * 32) * (T::NI * 32) + base + r % (IB * 32); };
  auto row = [&](int it) { return tile_row(r0 + it * kRowStep); };
  const char* in_hi = work + (kSym ? at_.p : q.xh);
  const char* in_lo = work + (WHAT == P_MUL ? at_.q : WHAT == P_POLY ? q.al : q.xl);
  const bool read_lo = WHAT != P_POLY || two;
  const bool step_rows = WHAT == P_STEP && !tall, whole_row = j + 8 <= n && n % 8 == 0;
  In8 in[2][kAhead];
  auto fetch = [&](int group) {
    if constexpr (WHAT != P_GRAM) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        In8& x = in[group & 1][u];
        const int i = min(row(group * kAhead + u), m - 1);   // rows past the end: any valid ones
        const int64_t at = (static_cast<int64_t>(i) * jp + min(j, jp - 8)) * 2;
        x.hi = *reinterpret_cast<const h8*>(in_hi + at);
        x.lo = h8{};
        if (read_lo) x.lo = *reinterpret_cast<const h8*>(in_lo + at);
        x.d = diag[i];
        if constexpr (WHAT == P_STEP) {
          if (step_rows && whole_row) {
            const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(out) + q.start + static_cast<int64_t>(i) * n + j);
            x.p[0] = p[0];
            x.p[1] = p[1];
          }
        }
      }
    }
  };
  fetch(0);
  float dj[8] = {};
  if constexpr (WHAT == P_POLY || WHAT == P_MUL) {
    const f32x4* d = reinterpret_cast<const f32x4*>(work + at_.dq + min(j, mp - 8) * 4);   // 256-byte padded: whole vectors
#pragma unroll
    for (int t = 0; t < 8; ++t) dj[t] = d[t / 4][t % 4];
  }
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int jj = 0; jj < T::NJ; ++jj)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int rr = wr * IB * 32 + i * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
        const int cc = wc * T::NJ * 32 + jj * 32 + lane % 32;
        stage[rr * BM + (cc ^ (4 * (rr / 8 % 16)))] = acc[i][jj][r];
      }
  __syncthreads();
  const bool mirror = kSym ? job.i != job.j : WHAT == P_APPLY || tall;
#pragma unroll
  for (int it = 0; it < kRows; ++it) {
    if (it % kAhead == 0 && it + kAhead < kRows) fetch(it / kAhead + 1);
    const In8& x = in[it / kAhead & 1][it % kAhead];
    const int r = r0 + kRowStep * it, i = row(it), sw = 4 * (r / 8 % 16);
    f32x4* s0 = reinterpret_cast<f32x4*>(stage + r * BM + (c ^ sw));
    f32x4* s1 = reinterpret_cast<f32x4*>(stage + r * BM + ((c + 4) ^ sw));
    float v[8];
#pragma unroll
    for (int t = 0; t < 4; ++t) { v[t] = (*s0)[t]; v[4 + t] = (*s1)[t]; }
    if constexpr (WHAT == P_GRAM) {
      const float g = kOpScale / (ex * ex);
#pragma unroll
      for (int t = 0; t < 8; ++t) v[t] *= g;
      if (job.i == job.j) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (i == j + t) {
            if (i < m) diag[i] = v[t] / kOpScale;
            v[t] = 0.0f;
          }
      }
    } else if constexpr (WHAT == P_POLY) {
      float* db = reinterpret_cast<float*>(work + at_.dout);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float a = static_cast<float>(x.hi[t]) + static_cast<float>(x.lo[t]) * (1.0f / kLowScale);
        const float a2 = v[t] * (1.0f / kOpScale);
        float y = k.b * a + k.c * (a2 + (x.d + dj[t]) * a);
        if (job.i == job.j && i == j + t) {
          const float rest = k.b * x.d + k.c * (a2 * (1.0f / kOpScale) + x.d * x.d);
          const bool all = x.d > 0.5f;
          if (i < m) db[i] = all ? k.a + rest : k.a;
          y = all ? 0.0f : rest * kOpScale;
        }
        v[t] = y;
      }
    } else if constexpr (WHAT == P_MUL) {
      float* dout = reinterpret_cast<float*>(work + at_.dout);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float y = v[t] * (1.0f / kOpScale) + (x.d * static_cast<float>(x.lo[t]) + static_cast<float>(x.hi[t]) * dj[t]);
        if (job.i == job.j && i == j + t) {
          const float full = y * (1.0f / kOpScale) + x.d * dj[t];
          // S: its diagonal as in a single step, by the row's length before both
          const float d = pair != kPairS || (i < m && reinterpret_cast<const float*>(work + q.da)[i] > 0.5f) ? full : k.a;
          if (i < m) dout[i] = d;
          y = (full - d) * kOpScale;
        }
        v[t] = y;
      }
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        v[t] = v[t] * (1.0f / kOpScale) +
               x.d * (static_cast<float>(x.hi[t]) + static_cast<float>(x.lo[t]) * (1.0f / kLowScale));
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = i < m && j + t < jn ? v[t] : 0.0f;
    if constexpr (!kLast) {
      if (i < m && j < jp) {
        h8 hi, lo;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          _Float16 a, b;
          split(v[t], a, b);
          hi[t] = a;
          lo[t] = b;
        }
        const int64_t at = (static_cast<int64_t>(i) * jp + j) * 2;
        *reinterpret_cast<h8*>(work + (kSym ? at_.out : q.xh) + at) = hi;
        if (WHAT == P_APPLY || (WHAT != P_MUL && two))
          *reinterpret_cast<h8*>(work + (WHAT == P_GRAM ? q.al : WHAT == P_POLY ? q.bl : q.xl) + at) = lo;
      }
    } else if (!tall && i < m && j < n) {
      finish(out, q.start + static_cast<int64_t>(i) * n + j, v, n - j, whole_row, f, k.decay, x.p);
    }
    if (mirror) {
      *s0 = f32x4{v[0], v[1], v[2], v[3]};
      *s1 = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
  if (!mirror) return;
  // column-wise: eight rows per thread, kHeight / 8 threads along a column
  const int cr = tid % (kHeight / 8) * 8, csw = 4 * (cr / 8 % 16), c0 = tid / (kHeight / 8);
  const int i = tile_row(cr);
  const bool whole_col = i + 8 <= m && m % 8 == 0;
  f32x4 p[2][2] = {};
  auto fetch_col = [&](int it) {
    if constexpr (WHAT == P_STEP) {
      const int jc = j0 + c0 + it * kColStep;
      if (whole_col && jc < n) {
        const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const float*>(out) + q.start + static_cast<int64_t>(jc) * m + i);
        p[it & 1][0] = s[0];
        p[it & 1][1] = s[1];
      }
    }
  };
  fetch_col(0);
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kCols; ++it) {
    if (it + 1 < kCols) fetch_col(it + 1);
    const int cc = c0 + it * kColStep, jc = j0 + cc;
    float v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = stage[(cr + t) * BM + (cc ^ csw)];
    if (jc >= jn) continue;
    if constexpr (!kLast) {
      if (i < mp) {
        h8 hi, lo;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          _Float16 a, b;
          split(v[t], a, b);
          hi[t] = a;
          lo[t] = b;
        }
        const int64_t at = (static_cast<int64_t>(jc) * mp + i) * 2;
        *reinterpret_cast<h8*>(work + at_.out + at) = hi;
        if (WHAT != P_MUL && two)
          *reinterpret_cast<h8*>(work + (WHAT == P_GRAM ? q.al : WHAT == P_POLY ? q.bl : q.xtl[at_.turn ^ 1]) + at) = lo;
      }
    } else if (i < m) {
      finish(out, q.start + static_cast<int64_t>(jc) * m + i, v, m - i, whole_col, f, k.decay, p[it & 1]);
    }
  }
}
};

// One job of one product.
template <int BM, Product WHAT>
__global__ __launch_bounds__(Tile<BM>::kNT) void mat_product_kernel(const MuonMat* __restrict__ mats,
                                                             const ProductJob* __restrict__ jobs, char* work,
                                                             int64_t slabs, int turn, int pair, MuonK k,
                                                             void* out) {
  using T = Tile<BM>;
  using St = Store<BM, WHAT, 2, T::IB>;
  static_assert(St::kBytes <= T::kLds, "a pass fits the operand stages");
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  const ProductJob job = jobs[blockIdx.x];
  const MuonMat& q = mats[job.mat];
  const int ld = WHAT == P_GRAM ? q.np : q.mp;
  const Where at = where<WHAT>(q, turn, pair);
  const char *p_hi = work + at.p, *q_hi = work + at.q;
  const char* p_lo = work + (WHAT == P_GRAM ? q.xl : WHAT == P_POLY ? q.al : q.bl);
  const char* q_lo = work + (WHAT == P_GRAM ? q.xl : WHAT == P_POLY ? q.al : q.xtl[at.turn]);
  const bool two = q.two_part;
  Acc<BM> acc = {};
  auto multiply = [&](const char* x, const char* y) {
    Multiply<BM>::run(reinterpret_cast<const _Float16*>(x), reinterpret_cast<const _Float16*>(y), ld, job.i * BM, q.m,
                      job.j * BM, St::kSym ? q.m : q.n, job.k0, job.k1, lds, acc);
  };
  if (two) {   // high * low + low * high, ahead of high * high
    for (int part = 0; part < 2; ++part) multiply(part ? p_lo : p_hi, part ? q_hi : q_lo);
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
      for (int j = 0; j < T::NJ; ++j) acc.v[i][j] *= 1.0f / kLowScale;
  }
  multiply(p_hi, q_hi);
  if (job.parts > 1) {
    Slab<BM>::store(acc, work + slabs, job.slab);
    return;
  }
#pragma unroll
  for (int pass = 0; pass < T::kPasses; ++pass) {
    if (pass) __syncthreads();
    St::run(reinterpret_cast<const f32x16 (&)[T::IB][T::NJ]>(acc.v[pass * T::IB]), job, q, pass * T::IB * 32, work, lds,
            turn, pair, k, out);
  }
}

// 32 rows of one cut tile: its parts' sums added up, then stored as above.
template <int BM, Product WHAT>
__global__ __launch_bounds__(Tile<BM>::WC * kWave) void mat_join_kernel(const MuonMat* __restrict__ mats,
                                                                        const ProductJob* __restrict__ joins,
                                                                        char* work, int64_t slabs, int turn, int pair,
                                                                        MuonK k, void* out) {
  using T = Tile<BM>;
  using St = Store<BM, WHAT, 1, 1>;
  __shared__ __attribute__((aligned(16))) char lds[St::kBytes];
  const ProductJob job = joins[blockIdx.x / (BM / 32)];
  const int strip = blockIdx.x % (BM / 32);
  const MuonMat& q = mats[job.mat];
  if (job.i * BM + strip * 32 >= q.mp) return;   // nothing of the matrix or its padding
  f32x16 v[1][T::NJ];
  Slab<BM>::add(v, work + slabs, job.slab, job.parts, strip);
  St::run(v, job, q, strip * 32, work, lds, turn, pair, k, out);
}

// ------------------------------------------------------------------ small matrices

// Matrices of at most 64 x 256 (X's sides), one workgroup each, whole call in
// one launch: what a step of three launches waits for is latency, and X fits
// LDS (64 x 48: 25 us, 104 us by launches). Every wave holds its part of X in
// fp32 registers, as the 16 x 16 blocks that v_mfma_f32_16x16x32_f16 gives; LDS
// holds the operands, high and low parts of X, X^T and of A or the polynomial.
// Products are high * low + low * high + high * high, and the polynomial's
// whole diagonal stays in fp32. Rows in LDS are 16 bytes longer than their
// contents, so that the rows of a fragment start in different banks.
constexpr int kTinyThreads = 512, kTinyWaves = kTinyThreads / kWave;
constexpr int kTinyM = static_cast<int>(kMatTinyM), kTinyN = static_cast<int>(kMatTinyN);
constexpr int kTinyBlocks = (kTinyM / 16) * (kTinyN / 16) / kTinyWaves;   // of X, per wave
typedef float f32v4 __attribute__((ext_vector_type(4)));

struct TinyLds {
  _Float16 x[2][kTinyM][kTinyN + 8];    // high, low
  _Float16 xt[2][kTinyN][kTinyM + 8];
  _Float16 a[2][kTinyM][kTinyM + 8];    // A, then the polynomial, without diagonal
  float da[kTinyM], db[kTinyM];
  double red[kTinyWaves];
};

// Sum over k of P[p0 + lane % 16][k] Q[q0 + ..][k], k < depth, both parts.
template <int LD>
__device__ __forceinline__ f32v4 tiny_product(const _Float16 (*P)[LD], const _Float16 (*Pl)[LD], int p0,
                                              const _Float16 (*Q)[LD], const _Float16 (*Ql)[LD], int q0, int depth,
                                              int lane) {
  f32v4 cross = {}, c = {};
  const int r = lane % 16, k0 = lane / 16 * 8;
  for (int k = k0; k < depth; k += 32) {
    const h8 p = *reinterpret_cast<const h8*>(&P[p0 + r][k]), pl = *reinterpret_cast<const h8*>(&Pl[p0 + r][k]);
    const h8 q = *reinterpret_cast<const h8*>(&Q[q0 + r][k]), ql = *reinterpret_cast<const h8*>(&Ql[q0 + r][k]);
    cross = __builtin_amdgcn_mfma_f32_16x16x32_f16(p, ql, cross, 0, 0, 0);
    cross = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, q, cross, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(p, q, c, 0, 0, 0);
  }
  return c + cross * (1.0f / kLowScale);
}

struct TinyCoeffs {
  float v[kMuonMaxSteps][3];
};

template <bool BF16, bool MUON>
__global__ __launch_bounds__(kTinyThreads) void mat_tiny_kernel(const MuonMat* __restrict__ mats, const void* grad,
                                                                float* mom, void* out, MuonK k, TinyCoeffs coeffs,
                                                                int steps, double eps) {
  __shared__ __attribute__((aligned(16))) TinyLds s;
  const MuonMat& q = mats[blockIdx.x];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int m = q.m, n = q.n, nb = (n + 15) / 16, depth = (n + 31) / 32 * 32;
  // this wave's blocks: rows bi * 16, columns (bj + 2 b) * 16; this lane's
  // elements of a block: rows i .. i + 3, column j
  const int bi = wave % 4, bj = wave / 4, i = bi * 16 + lane / 16 * 4;
  auto col = [&](int b) { return (bj + 2 * b) * 16 + lane % 16; };
  auto at = [&](int r, int j) { return q.start + (q.tall ? static_cast<int64_t>(j) * m + i + r : static_cast<int64_t>(i + r) * n + j); };
  float x[kTinyBlocks][4];
  double sum = 0.0;
#pragma unroll
  for (int b = 0; b < kTinyBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[b][r] = 0.0f;
      if (i + r < m && col(b) < n) {
        const int64_t e = at(r, col(b));
        float g = load_elem(grad, e, BF16);
        if constexpr (MUON) {
          const float mm = __fadd_rn(__fmul_rn(k.mu, mom[e]), g);
          mom[e] = mm;
          g = k.nesterov ? __fadd_rn(g, __fmul_rn(k.mu, mm)) : mm;
        }
        x[b][r] = g;
        sum += static_cast<double>(g) * static_cast<double>(g);
      }
    }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if (lane == 0) s.red[wave] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < kTinyWaves; ++w) sum += s.red[w];
  const float ex = static_cast<float>(1 << q.ex);
  const double inv = static_cast<double>(ex) / (sqrt(sum) + eps);
  auto put_x = [&]() {
#pragma unroll
    for (int b = 0; b < kTinyBlocks; ++b) {
      if ((bj + 2 * b) * 16 >= depth) break;
      _Float16 h[4], l[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        split(x[b][r], h[r], l[r]);
        s.x[0][i + r][col(b)] = h[r];
        s.x[1][i + r][col(b)] = l[r];
      }
      typedef _Float16 h4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<h4*>(&s.xt[0][col(b)][i]) = h4{h[0], h[1], h[2], h[3]};
      *reinterpret_cast<h4*>(&s.xt[1][col(b)][i]) = h4{l[0], l[1], l[2], l[3]};
    }
  };
#pragma unroll
  for (int b = 0; b < kTinyBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) x[b][r] = static_cast<float>(static_cast<double>(x[b][r]) * inv);
  put_x();
  for (int t = 0; t < steps; ++t) {
    const float ca = coeffs.v[t][0], cb = coeffs.v[t][1], cc = coeffs.v[t][2];
    __syncthreads();
    // A: blocks (bi, bj) and (bi, bj + 2)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j = col(b);
      const f32v4 v = tiny_product(s.x[0], s.x[1], bi * 16, s.x[0], s.x[1], (bj + 2 * b) * 16, depth, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float y = v[r] * (kOpScale / (ex * ex));
        if (i + r == j) {
          s.da[j] = y / kOpScale;
          y = 0.0f;
        }
        split(y, s.a[0][i + r][j], s.a[1][i + r][j]);
      }
    }
    __syncthreads();
    float y[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j = col(b);
      const f32v4 v = tiny_product(s.a[0], s.a[1], bi * 16, s.a[0], s.a[1], (bj + 2 * b) * 16, kTinyM, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float a = static_cast<float>(s.a[0][i + r][j]) + static_cast<float>(s.a[1][i + r][j]) * (1.0f / kLowScale);
        const float di = s.da[i + r], a2 = v[r] * (1.0f / kOpScale);
        y[b][r] = cb * a + cc * (a2 + (di + s.da[j]) * a);
        if (i + r == j) {
          s.db[j] = ca + cb * di + cc * (a2 * (1.0f / kOpScale) + di * di);
          y[b][r] = 0.0f;
        }
      }
    }
    __syncthreads();   // A is read
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) split(y[b][r], s.a[0][i + r][col(b)], s.a[1][i + r][col(b)]);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kTinyBlocks; ++b) {
      if (bj + 2 * b >= nb) break;
      const f32v4 v = tiny_product(s.a[0], s.a[1], bi * 16, s.xt[0], s.xt[1], (bj + 2 * b) * 16, kTinyM, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[b][r] = v[r] * (1.0f / kOpScale) + s.db[i + r] * x[b][r];
    }
    if (t + 1 == steps) break;
    __syncthreads();   // X and X^T are read
    put_x();
  }
  const float f = MUON ? k.lr * update_scale(k.scale_mode, q.rows, q.cols) / ex : 1.0f / ex;
#pragma unroll
  for (int b = 0; b < kTinyBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (i + r < m && col(b) < n) {
        const int64_t e = at(r, col(b));
        if constexpr (MUON) {
          float* p = static_cast<float*>(out);
          p[e] = __fsub_rn(__fmul_rn(p[e], k.decay), __fmul_rn(f, x[b][r]));
        } else {
          static_cast<uint16_t*>(out)[e] = static_cast<uint16_t>(bf16_rne(x[b][r] * f));
        }
      }
    }
}

// ------------------------------------------------------------------ launches

template <int BM, Product WHAT>
void launch_tiles(const rs_plan* p, int list, char* work, int turn, int pair, const MuonK& k, void* out, hipStream_t s) {
  hipLaunchKernelGGL((mat_product_kernel<BM, WHAT>), dim3(static_cast<unsigned>(p->n_mat_jobs[list])),
                     dim3(Tile<BM>::kNT), 0, s, p->mats, p->mat_jobs[list], work, p->mat_slabs, turn, pair, k, out);
  if (p->n_mat_joins[list])
    hipLaunchKernelGGL((mat_join_kernel<BM, WHAT>),
                       dim3(static_cast<unsigned>(p->n_mat_joins[list] * (BM / 32))), dim3(Tile<BM>::WC * kWave), 0, s,
                       p->mats, p->mat_joins[list], work, p->mat_slabs, turn, pair, k, out);
}

template <Product WHAT>
void launch_product(const rs_plan* p, int list, char* work, int turn, int pair, const MuonK& k, void* out, hipStream_t s) {
  if (p->n_mat_jobs[list] == 0) return;
  if (p->mat_side[list] == 256) launch_tiles<256, WHAT>(p, list, work, turn, pair, k, out, s);
  else if (p->mat_side[list] == 128) launch_tiles<128, WHAT>(p, list, work, turn, pair, k, out, s);
  else launch_tiles<64, WHAT>(p, list, work, turn, pair, k, out, s);
}

// Momentum (MUON), norm and Newton-Schulz on every matrix of the plan; the
// last product writes `out` (bf16 values, or fp32 parameters in place).
template <bool MUON>
int run_matrices(rs_plan* p, const void* grad, int32_t grad_dt, float* mom, const float* coeffs, int32_t steps,
                 float eps, MuonK k, void* out, char* work, hipStream_t s, const char* who) {
  if (p->n_tiny) {
    TinyCoeffs c{};
    std::copy(coeffs, coeffs + 3 * steps, &c.v[0][0]);
    const dim3 grid(static_cast<unsigned>(p->n_tiny));
    if (grad_dt == RS_BF16)
      hipLaunchKernelGGL((mat_tiny_kernel<true, MUON>), grid, dim3(kTinyThreads), 0, s, p->tiny, grad, mom, out, k, c,
                         steps, static_cast<double>(eps));
    else
      hipLaunchKernelGGL((mat_tiny_kernel<false, MUON>), grid, dim3(kTinyThreads), 0, s, p->tiny, grad, mom, out, k, c,
                         steps, static_cast<double>(eps));
  }
  if (p->n_mats == 0) return launched(who);
  const dim3 chunks(static_cast<unsigned>(p->n_mat_chunks)), spread(static_cast<unsigned>(p->n_mat_spread));
  if (grad_dt == RS_BF16) {
    hipLaunchKernelGGL((mat_norm_kernel<true, MUON>), chunks, dim3(kThreads), 0, s, p->mats, p->mat_chunks, grad, mom,
                       work, k);
  } else {
    hipLaunchKernelGGL((mat_norm_kernel<false, MUON>), chunks, dim3(kThreads), 0, s, p->mats, p->mat_chunks, grad, mom,
                       work, k);
  }
  const bool own_scale = p->mat_own_scale;
  if (!own_scale)
    hipLaunchKernelGGL(mat_scale_kernel, dim3(static_cast<unsigned>(p->n_mats)), dim3(kThreads), 0, s, p->mats, work,
                     static_cast<double>(eps));
  if (grad_dt == RS_BF16) {
    hipLaunchKernelGGL((mat_spread_kernel<true, MUON>), spread, dim3(kThreads), 0, s, p->mats, p->mat_spread, grad,
                       mom, work, k, own_scale, static_cast<double>(eps));
  } else {
    hipLaunchKernelGGL((mat_spread_kernel<false, MUON>), spread, dim3(kThreads), 0, s, p->mats, p->mat_spread, grad,
                       mom, work, k, own_scale, static_cast<double>(eps));
  }
  auto polynomial = [&](int t) {
    k.a = coeffs[3 * t];
    k.b = coeffs[3 * t + 1];
    k.c = coeffs[3 * t + 2];
  };
  auto apply = [&](int list, int t, int pair) {
    if (t + 1 < steps) launch_product<P_APPLY>(p, list, work, t, pair, k, nullptr, s);
    else launch_product<MUON ? P_STEP : P_OUT>(p, list, work, t, pair, k, out, s);
  };
  const bool pairs = p->mat_any_paired && steps >= 2 && std::fabs(coeffs[0]) <= kPairMaxA && std::fabs(coeffs[3]) <= kPairMaxA;
  if (pairs) {
    polynomial(0);
    launch_product<P_GRAM>(p, kGram, work, 0, 0, k, nullptr, s);
    launch_product<P_POLY>(p, kSquare, work, 0, 0, k, nullptr, s);
    launch_product<P_MUL>(p, kSquarePaired, work, 0, kPairT, k, nullptr, s);
    launch_product<P_MUL>(p, kSquarePaired, work, 0, kPairA1, k, nullptr, s);
    apply(kApplySingle, 0, 0);
    launch_product<P_GRAM>(p, kGramSingle, work, 0, 0, k, nullptr, s);
    polynomial(1);
    launch_product<P_POLY>(p, kSquare, work, 0, 1, k, nullptr, s);
    k.a = coeffs[0] * coeffs[3];
    launch_product<P_MUL>(p, kSquarePaired, work, 0, kPairS, k, nullptr, s);
    apply(kApply, 1, 1);
  }
  for (int t = pairs ? 2 : 0; t < steps; ++t) {
    polynomial(t);
    launch_product<P_GRAM>(p, kGram, work, t, 0, k, nullptr, s);
    launch_product<P_POLY>(p, kSquare, work, t, 0, k, nullptr, s);
    apply(kApply, t, pairs ? 0 : -1);   // -1: no matrix has two steps as one
  }
  return launched(who);
}

int check_matrices(const rs_plan* p, const float* coeffs, int32_t steps, float eps, const void* work,
                   int64_t work_bytes, const char* who) {
  if (p->mat_too_large)
    return fail(RS_ERANGE, std::string(who) + ": a WHOLE matrix has a side over " + std::to_string(kMatMaxSide) +
                               " or both over " + std::to_string(kMatMaxMin) + ", or there are too many");
  if (!coeffs || steps < 1 || steps > kMuonMaxSteps)
    return fail(RS_EINVAL, std::string(who) + ": 1 to " + std::to_string(kMuonMaxSteps) + " steps of three coefficients");
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(coeffs[i])) return fail(RS_EINVAL, std::string(who) + ": coefficients must be finite");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(RS_EINVAL, std::string(who) + ": eps must be finite and >= 0");
  if (p->mat_work_bytes && !work) return fail(RS_EINVAL, std::string(who) + ": null workspace");
  if (!aligned16(work)) return fail(RS_EALIGN, std::string(who) + ": workspace must be 16-byte aligned");
  if (work_bytes < p->mat_work_bytes)
    return fail(RS_EINVAL, std::string(who) + ": workspace of " + std::to_string(work_bytes) + " bytes, " +
                               std::to_string(p->mat_work_bytes) + " needed");
  return RS_OK;
}

}  // namespace
}  // namespace rs

using namespace rs;

extern "C" int rs_muon_workspace(const rs_plan* p, int64_t* bytes) {
  clear_error();
  if (!p || !bytes) return fail(RS_EINVAL, "rs_muon_workspace: null argument");
  *bytes = p->mat_work_bytes;
  return RS_OK;
}

extern "C" int rs_orthogonalize(rs_plan* p, const void* src, int32_t src_dt, void* out, const float* coeffs,
                                int32_t steps, float eps, void* work, int64_t work_bytes, void* stream) {
  const char* who = "rs_orthogonalize";
  clear_error();
  int st = check_call(p, who);
  if (st != RS_OK) return st;
  if (!src || !out) return fail(RS_EINVAL, std::string(who) + ": null argument");
  if (src_dt != RS_F32 && src_dt != RS_BF16) return fail(RS_EDTYPE, std::string(who) + ": src is fp32 or bf16");
  st = check_matrices(p, coeffs, steps, eps, work, work_bytes, who);
  if (st != RS_OK) return st;
  if (!aligned16(src) || !aligned16(out)) return fail(RS_EALIGN, std::string(who) + ": buffers must be 16-byte aligned");
  if (p->n_mats + p->n_tiny == 0) return RS_OK;
  return run_matrices<false>(p, src, src_dt, nullptr, coeffs, steps, eps, MuonK{}, out, static_cast<char*>(work),
                             static_cast<hipStream_t>(stream), who);
}

extern "C" int rs_muon_step(rs_plan* p, float* param, const void* grad, int32_t grad_dt, float* momentum,
                            const rs_muon_hparams* hp, const float* coeffs, void* work, int64_t work_bytes,
                            void* stream) {
  const char* who = "rs_muon_step";
  clear_error();
  int st = check_call(p, who);
  if (st != RS_OK) return st;
  if (!param || !grad || !momentum || !hp) return fail(RS_EINVAL, std::string(who) + ": null argument");
  if (grad_dt != RS_F32 && grad_dt != RS_BF16) return fail(RS_EDTYPE, std::string(who) + ": grad is fp32 or bf16");
  if (!std::isfinite(hp->lr) || !(hp->momentum >= 0.0f && hp->momentum < 1.0f) || !std::isfinite(hp->weight_decay) ||
      (hp->nesterov != 0 && hp->nesterov != 1) || hp->scale_mode < RS_MUON_SCALE_NONE ||
      hp->scale_mode > RS_MUON_SCALE_RMS)
    return fail(RS_EINVAL, std::string(who) + ": bad hyper-parameters");
  st = check_matrices(p, coeffs, hp->steps, hp->eps, work, work_bytes, who);
  if (st != RS_OK) return st;
  if (!aligned16(param) || !aligned16(grad) || !aligned16(momentum))
    return fail(RS_EALIGN, std::string(who) + ": buffers must be 16-byte aligned");
  if (p->n_mats + p->n_tiny == 0) return RS_OK;
  MuonK k{};
  k.mu = hp->momentum;
  k.lr = hp->lr;
  k.decay = static_cast<float>(1.0 - static_cast<double>(hp->lr) * static_cast<double>(hp->weight_decay));
  k.nesterov = hp->nesterov;
  k.scale_mode = hp->scale_mode;
  return run_matrices<true>(p, grad, grad_dt, momentum, coeffs, hp->steps, hp->eps, k, param, static_cast<char*>(work),
                            static_cast<hipStream_t>(stream), who);
}
