// The vocabulary head's losses with the head's table read from the gathered
// flat buffer and its gradient written into the packed one, on gfx950: kernels
// and the rs_head_loss / rs_head_grad / rs_distill_loss / rs_distill_grad /
// rs_head_workspace entry points ("veScale-FSDP: flexible, structure-aware
// sharding at 10K-GPU scale", feynmanwiki walkthrough, DBuffer paragraphs: a
// tensor is its planned slice, and scale / add / zero ahead of the reduction).
//
// Mathematics. With W the table (V rows of H columns), x_t a token's hidden
// state, c the factor on the logits and q_t the wanted distribution (one row of
// the table, or the softmax of a teacher's top logits):
//   l_t = c W x_t,  Z_t = log sum exp l_t,  p_t = exp(l_t - Z_t)
//   loss_t = f (sum_k q_k log q_k + Z_t - sum_k q_k l_k)
// and with d_t = p_t - q_t and a_t = weight_t f c, the gradients of
// sum weight_t loss_t:
//   dx_t = a_t W^T d_t,   dW = sum_t a_t d_t x_t^T.
// These are three products; nothing is computed twice. Tokens are taken in
// pieces: a piece's logits are stored (fp32) with each row's running maximum
// and sum per 128 columns, become d in place, and are used up by the piece's two
// gradient products. The maximum and the logarithm of the sum stay two numbers:
// log p is a logit's distance from the first less the second, as exact for logits
// of 100 as for those of 1. Tokens without a target take part in none of them: the
// others are brought together first.
//
// Number formats. The logits' product takes the bf16 operands as they are, with
// fp32 sums. d is computed in fp32 and rounded once for each of the two
// products that read it: to bf16 for dx, whose result is bf16 too and whose
// other operand is the table as gathered (range of bf16, no copy; what the
// rounding leaves at the targets is added by itself in fp32, all other rows keep
// 8 bits); to fp16, eight times finer, for dW, with x scaled to fp16 by a power of
// two. Where the packed buffer is fp32, a d has a second fp16 part that holds the
// rest of the first, and its product comes ahead of the first's: 22 bits, as near
// as fp32 products' for a d down to 2^-17 of the largest a. One scale serves the
// whole call, so smaller ones are rounded to within 2^-38 of the largest a
// (10 bits at 2^-29 of it, 0 below 2^-40), and x to within 2^-38 of the largest x.
#include "host_common.h"
#include "mfma.h"

#include <type_traits>

namespace rs {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kTileM = 256;          // rows of an output tile: its contiguous dimension in memory
constexpr int kStep = 64;            // of the contraction, per stage; what it is padded to
constexpr int kPart = 64;            // columns of d whose fp16 parts lie beside each other
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// ------------------------------------------------------------------ products

// C[m, n] = sum_k P[m, k] Q[n, k] on one 256 x BN tile, 32 x 32 accumulators. Either operand may lie with k contiguous (plain) or with its
// other index contiguous (TR): a TR operand is read out of LDS transposed
// (ds_read_b64_tr_b16), so the table and d are used as they lie in memory.
template <int BN, int WAVES = 8>
struct HeadTile {
  static constexpr int kN = BN, kWaves = WAVES, kThreads = kWaves * kWave;
  static constexpr int WR = BN == 256 ? 2 : 4;              // wave rows
  static constexpr int WC = kWaves / WR;
  static constexpr int NI = kTileM / 32 / WR, NJ = BN / 32 / WC;
  static constexpr int kStages = BN == 256 ? 2 : BN == 128 ? 3 : 4, kStagesQ = BN == 256 ? 3 : kStages;
  static constexpr int kLds = (kStages * kTileM + kStagesQ * BN) * kStep * 2;
};
// dx has four waves, which read less out of LDS for as many multiplications
// (2048 x 131072 x 2048: 0.85 ms, with eight 0.91); dW eight (4096 x 131072 x 4096
// with both parts: 6.9 ms, with four 8.0). The logits have eight, of which one
// multiplies while the other keeps its results, up to kShortCols columns, and four
// above (2048 tokens by 131072 rows of 256, 1024, 2048: 200, 549, 1060 us with eight,
// 270, 600, 1120 with four; 4096 tokens, 4096 columns: 3.86 ms and 3.74).
constexpr int64_t kShortCols = 2048;
template <int BN>
using DxTile = HeadTile<BN, BN == 256 ? 4 : 8>;
using DwTile = HeadTile<256>;

// One operand's tile: from `base` on, `left` bytes may be read. Plain: `rows`
// rows exist (those past them repeat the last), a stage lies `step` bytes behind
// the one ahead of it, and the contraction is padded.
// TR: `rows` values of k exist, at least one (those past them repeat the last:
// the other operand holds zeros there). PARTS: see Fetch.
struct Operand {
  const char* base;
  int64_t left;
  int pitch, rows;
  int64_t step;
};

// Memory to LDS, 16 bytes per lane and load. Plain: 128-byte rows, piece c of
// row r at place c ^ (r / 2 % 8). TR: rows of SIDE values, one per k, piece c of
// row k at place c ^ (4 * (k % 4)), so that the four rows that 32 lanes of a
// transposed read touch fall into banks of their own.
//   RAGGED: a TR operand's rows may end within a stage, or ahead of one.
//   PARTS: the operand is the fp16 parts of d, kPart columns of each beside each
// other.
template <int SIDE, bool TR, bool RAGGED, bool PARTS, int WAVES>
struct Fetch {
  static constexpr int kBytes = SIDE * kStep * 2;
  static constexpr int kLoads = kBytes / 1024 / WAVES;
  static constexpr int kRowLanes = TR ? SIDE / 8 : 8;        // lanes that load one row
  static_assert(kLoads * 1024 * WAVES == kBytes, "whole loads");
  int off[kLoads], wave, lane;

  __device__ __forceinline__ int row(int t) const { return (t * WAVES + wave) * (kWave / kRowLanes) + lane / kRowLanes; }
  __device__ __forceinline__ int piece(int r) const {
    const int c = (lane % kRowLanes) ^ (TR ? 4 * (r % 4) : r / 2 % 8);
    return PARTS ? c / 8 * 256 + c % 8 * 16 : c * 16;
  }
  __device__ __forceinline__ void init(const Operand& o) {
#pragma unroll
    for (int t = 0; t < kLoads; ++t) {
      const int r = row(t);
      off[t] = (TR ? r : min(r, o.rows - 1)) * o.pitch + piece(r);
    }
  }
  // Stage k of the contraction: loads [first, last) of this wave. `more`: bytes
  // that all of the operand lies further on.
  template <int FIRST, int LAST>
  __device__ __forceinline__ void load(const Operand& o, int k, int64_t more, lds_char* dst) const {
    if constexpr (FIRST < LAST) {
      const int first = RAGGED ? min(k * kStep, o.rows - 1) : k * kStep;
      const int64_t at = more + (TR ? static_cast<int64_t>(first) * o.pitch : k * o.step);
      const int64_t left = o.left - at;
      const __amdgpu_buffer_rsrc_t rsrc =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(o.base + at), 0,
                                            static_cast<int>(left < 0x7fffffff ? left : 0x7fffffff), kRawBufferWord3);
#pragma unroll
      for (int t = FIRST; t < LAST; ++t) {
        const int r = row(t);
        const int mine = RAGGED ? min(r, o.rows - 1 - first) * o.pitch + piece(r) : off[t];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, dst + (t * WAVES + wave) * 1024, 16, mine, 0, 0, 0);
      }
    }
  }
};

// A transposed read. The pointer is marked as aliasing nothing else: otherwise
// the compiler waits for every load into LDS on its way ahead of each read,
// where the contraction waits for the one stage that it reads.
__device__ __forceinline__ u32x2 read_tr(const lds_s16x4* __restrict__ p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<lds_s16x4*>(p)));
}

// LDS to fragments: 32 rows (m or n) by 16 k, lane l has row l % 32 and the 8
// values of k from 8 * (l / 32) on. A transposed read gives each lane of 16 the
// column of its number of a 4 x 16 block, so a fragment takes two.
template <int SIDE, bool TR, int N>
struct Fragments {
  static constexpr int kBytes = SIDE * kStep * 2;
  const char* at[TR ? N : kStep / 16];

  __device__ __forceinline__ void init(const char* lds, int first, int lane) {   // first: the wave's first 32-row block
    if constexpr (TR) {
      const int i = lane % 16, g = lane / 16, k = g / 2 * 8 + i / 4;
#pragma unroll
      for (int b = 0; b < N; ++b) {
        const int piece = (first + b) * 4 + g % 2 * 2 + i % 4 / 2;
        at[b] = lds + k * SIDE * 2 + (piece ^ (4 * (k % 4))) * 16 + i % 2 * 8;
      }
    } else {
      const int r = lane % 32;
#pragma unroll
      for (int kk = 0; kk < kStep / 16; ++kk) at[kk] = lds + first * 4096 + r * 128 + ((kk * 2 + lane / 32) ^ (r / 2 % 8)) * 16;
    }
  }
  __device__ __forceinline__ u32x4 read(int b, int kk, int stage) const {
    if constexpr (TR) {
      const char* p = at[b] + stage * kBytes + kk * 16 * SIDE * 2;
      const u32x2 a = read_tr((const lds_s16x4*)(const lds_char*)p), c = read_tr((const lds_s16x4*)(const lds_char*)(p + 4 * SIDE * 2));
      return u32x4{a.x, a.y, c.x, c.y};
    } else {
      return *reinterpret_cast<const u32x4*>(at[kk] + stage * kBytes + b * 4096);
    }
  }
};

template <class T>
struct HeadAcc {
  f32x16 v[T::NI][T::NJ];
};

// The contraction, in `ksteps` stages. With `two`, after the first half of them
// P starts over and Q starts over at its other part, `second` bytes further on.
//   One stage: sixteen-column multiplications, each while the next fragment is
// read; then, with every wave done reading this stage and the next one arrived,
// the last of them under the first reads of the next stage. From there
// on, spread over a whole stage, the places that this stage leaves are loaded
// again, P's for kStages stages later and behind them Q's for kStagesQ later.
// A load into LDS holds its wave up while others are on their way, so loads in
// one burst stop the multiplications: in one, dx of 4096 x 131072 x 4096 took
// 3.84 ms, spread it takes 3.0 to 3.2 (1370 to 1460 TFLOP/s, the matrix cores busy
// for 83% of it at 1.55 to 1.6 GHz; a library product of the size 2.8). For the
// logits they are busy 66 to 74%, for dW 75 to 78%, at 1.5 to 1.7 GHz.
template <class T, bool F16, bool PT, bool QT, bool RAGGED, bool PARTS>
struct Contract {
using FP = Fetch<kTileM, PT, RAGGED, false, T::kWaves>;
using FQ = Fetch<T::kN, QT, false, PARTS, T::kWaves>;
static constexpr int kParts = kStep / 16;   // multiplications of a stage, and parts of its loads
static constexpr int SP = T::kStages, SQ = T::kStagesQ, U = SP == SQ ? SP : SP * SQ;
static constexpr int LP = FP::kLoads, LQ = FQ::kLoads, kLoads = LP + LQ;
static constexpr int kReads = T::NI * (PT ? 2 : 1) + T::NJ * (QT ? 2 : 1), kMuls = T::NI * T::NJ;
static_assert(SQ == SP || SQ == SP + 1, "the counts of loads on their way below");

Operand p, q;
int ksteps, turn;
int64_t second;
lds_char* base;
FP fp;
FQ fq;
Fragments<kTileM, PT, T::NI> rp;
Fragments<T::kN, QT, T::NJ> rq;
u32x4 fa[2][T::NI], fb[2][T::NJ];

template <int FIRST, int LAST>
__device__ __forceinline__ void load_p(int s, int place) {
  fp.template load<FIRST, LAST>(p, s < turn ? s : s - turn, 0, base + place * FP::kBytes);
}
template <int FIRST, int LAST>
__device__ __forceinline__ void load_q(int s, int place) {
  fq.template load<FIRST, LAST>(q, s < turn ? s : s - turn, s < turn ? 0 : second, base + SP * FP::kBytes + place * FQ::kBytes);
}
// Part PART of what is loaded into the places of stage s.
template <int PART>
__device__ __forceinline__ void load_part(int s, int pp, int qp, bool whole) {
  constexpr int a = kLoads * PART / kParts, b = kLoads * (PART + 1) / kParts;
  if (whole || s + SP < ksteps) load_p<(a < LP ? a : LP), (b < LP ? b : LP)>(s + SP, pp);
  if (whole || s + SQ < ksteps) load_q<(a > LP ? a - LP : 0), (b > LP ? b - LP : 0)>(s + SQ, qp);
}
__device__ __forceinline__ void fetch(int pp, int qp, int kk, int to) {
#pragma unroll
  for (int j = 0; j < T::NJ; ++j) fb[to][j] = rq.read(j, kk, qp);
#pragma unroll
  for (int i = 0; i < T::NI; ++i) fa[to][i] = rp.read(i, kk, pp);
}
__device__ __forceinline__ void mma(HeadAcc<T>& c, int from) {
#pragma unroll
  for (int i = 0; i < T::NI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) {
      if constexpr (F16)
        c.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, fa[from][i]), __builtin_bit_cast(h8, fb[from][j]),
                                                           c.v[i][j], 0, 0, 0);
      else
        c.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, fa[from][i]), __builtin_bit_cast(b8, fb[from][j]),
                                                            c.v[i][j], 0, 0, 0);
    }
}
// Multiplications with the fragment reads between them, and behind the reads
// the LOADS loads.
template <int LOADS>
__device__ static __forceinline__ void interleave() {
  constexpr int kEach = (kReads + kMuls - 1) / kMuls, kRead = (kReads + kEach - 1) / kEach;
  constexpr int kRest = kMuls > kRead ? kMuls - kRead : 1, kLoadEach = (LOADS + kRest - 1) / kRest;
#pragma unroll
  for (int i = 0; i < kMuls; ++i) {
    if (i < kRead) __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);   // LDS reads
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                      // one multiplication
    if (LOADS && (i >= kRead || i == kMuls - 1)) __builtin_amdgcn_sched_group_barrier(0x020, kLoadEach, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}
template <int KK>
__device__ __forceinline__ void sixteen(HeadAcc<T>& c, int s, int pp, int qp, int before_p, int before_q, bool whole) {
  fetch(pp, qp, KK + 1, (KK + 1) & 1);
  if (whole || s > 0) load_part<KK + 1>(s - 1, before_p, before_q, whole);
  mma(c, KK & 1);
  interleave<kLoads * (KK + 2) / kParts - kLoads * (KK + 1) / kParts>();
}
// Stage s, in places pp and qp; before_p, before_q: those of stage s - 1.
// whole: everything that a stage loads exists, and stages ahead of this one.
__device__ __forceinline__ void step(HeadAcc<T>& c, int s, int pp, int qp, int next_p, int next_q, int before_p, int before_q, bool whole) {
  sixteen<0>(c, s, pp, qp, before_p, before_q, whole);
  sixteen<1>(c, s, pp, qp, before_p, before_q, whole);
  sixteen<2>(c, s, pp, qp, before_p, before_q, whole);
  // newer than the next stage's loads: SP - 2 turns' and Q's of one stage more
  if (whole || s + SQ <= ksteps) wait<(SP - 2) * kLoads + (SQ - SP) * LQ, true>();
  else wait<0, true>();
  barrier();
  if (whole || s + 1 < ksteps) fetch(next_p, next_q, 0, 0);
  load_part<0>(s, pp, qp, whole);
  mma(c, 1);
  interleave<kLoads / kParts>();
}

__device__ __forceinline__ explicit Contract(char* lds) : base((lds_char*)lds) {
  const int tid = fresh_thread(), lane = tid % kWave;
  fp.wave = fq.wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  fp.lane = fq.lane = lane;
  rp.init(lds, fp.wave / T::WC * T::NI, lane);
  rq.init(lds + SP * FP::kBytes, fp.wave % T::WC * T::NJ, lane);
}

// The first stages' loads of a tile. Every wave has left the loop of run for
// the tile ahead of it, which is done with LDS then, so a tile's loads can be
// on their way while the one ahead of it is stored.
__device__ __forceinline__ void begin(const Operand& p_, const Operand& q_, int ksteps_, bool two, int64_t second_) {
  p = p_;
  q = q_;
  ksteps = ksteps_;
  turn = two ? ksteps / 2 : ksteps;
  second = second_;
  fp.init(p);
  fq.init(q);
#pragma unroll
  for (int s = 0; s < SQ; ++s) {
    if (s < SP && s < ksteps) load_p<0, LP>(s, s);
    if (s < ksteps) load_q<0, LQ>(s, s);
  }
}

// c <- the contraction. ahead: what has been loaded or stored since begin is
// counted as well, so all of it has to arrive.
__device__ __forceinline__ void run(HeadAcc<T>& c, bool ahead) {
#pragma unroll
  for (int i = 0; i < T::NI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) c.v[i][j] = f32x16{};
  if (ksteps == 0) return;
  if (!ahead && ksteps >= SQ) wait<(SP - 1) * kLoads + (SQ - SP) * LQ, false>();
  else wait<0, false>();
  barrier();
  fetch(0, 0, 0, 0);
  int s = 0;
  if (ksteps > 2 * U) {   // the first has no stage ahead of it
    step(c, 0, 0, 0, 1 % SP, 1 % SQ, 0, 0, false);
    for (s = 1; s + U - 1 + SQ < ksteps; s += U) {
#pragma unroll
      for (int u = 1; u <= U; ++u)
        step(c, s + u - 1, u % SP, u % SQ, (u + 1) % SP, (u + 1) % SQ, (u - 1) % SP, (u - 1) % SQ, true);
    }
  }
  for (; s < ksteps; ++s) step(c, s, s % SP, s % SQ, (s + 1) % SP, (s + 1) % SQ, (s + SP - 1) % SP, (s + SQ - 1) % SQ, false);
}
};

// Tile number `o` of m_tiles x n_tiles, eight m tiles beside each other within
// a band, so that the 32 neighbours that an XCD's CUs work on at a time share
// operands in its L2.
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int o, int across, int along, bool m_across) {
  constexpr int kBand = 8;
  const int band = o / (kBand * along), rest = o - band * kBand * along;
  const int wide = min(kBand, across - band * kBand);
  const int a = band * kBand + rest % wide, b = rest / wide;
  return m_across ? TileAt{a, b} : TileAt{b, a};
}

// The work items of this workgroup out of n: workgroup b runs on XCD b % 8, and
// each XCD takes a contiguous eighth, its workgroups in turn.
struct Items {
  int now, end, stride;
  __device__ __forceinline__ explicit Items(int n) {
    const int per = (n + 7) / 8, xcd = static_cast<int>(blockIdx.x) % 8;
    now = xcd * per + static_cast<int>(blockIdx.x) / 8;
    end = min((xcd + 1) * per, n);
    stride = static_cast<int>(gridDim.x) / 8;
  }
};

// ------------------------------------------------------------------ call

// What the tokens of a call come to, known on the device only.
struct HeadInfo {
  int32_t count;     // tokens with a target
  int32_t ex, ec;    // |a_t| < 2^ec over them, |x| < 2^ex over those of a_t that is not 0
  int32_t pad;
};
struct HeadPiece {
  int32_t count;     // of this piece's tokens
  int32_t splits;    // of the contraction of dx
};

// A call as the kernels see it. Kept tokens are numbered 0.. count-1 in their
// own order; arrays "by token" have n entries, arrays "by place" have npad.
struct Head {
  int32_t n, npad, rows, cols, vp, hp, top, piece;   // vp, hp: rows and columns padded
  const char* table;      // bf16, pitch bytes a row
  int32_t pitch;
  int64_t table_bytes;
  HeadInfo* info;
  HeadPiece* pieces;
  uint32_t* keep;         // by token: has a target
  float *xmax, *ent;      // by token: largest finite |x|, sum q log q
  int32_t* idx;           // by token, top each, ascending: row of the table, kNone behind them
  float* q;
  int32_t* kept;          // by place: the token
  float *pent, *a;        // by place
  float2* lse;            // by place, in powers of two: the largest logit, log of the sum of exponentials ahead of it
  int32_t* pidx;          // by place, top each: the same
  float *pq, *picked;     // q and the logit there
  char *xb, *xh;          // by place: x in bf16, 64 columns of all tokens beside each other, and scaled in fp16, 256 columns
  float2* stat;           // of one piece: per 32 * NI rows of the table, `piece` maxima and sums
  float* logits;          // of one piece: see logit_at; then the fp16 parts of d, 256 columns of all its tokens beside each other
  uint16_t* d;            // of one piece: bf16, 64 columns of all its tokens beside each other
  char* slabs;
  float* rest;            // what rounding left of d at the targets
  float* fix;             // of one piece: its share of dx, hp columns a token
};

// ------------------------------------------------------------------ targets

constexpr int kMaxTop = 256;
constexpr int kNone = 0x7fffffff;   // behind every row of the table

// One token a wave: its rows of the table in ascending order and their share q,
// whether it has any, and the largest finite |x| (GRAD). A token without a target gets its
// loss (and dx) of zero here, and its x is not read.
template <bool GRAD>
__global__ __launch_bounds__(kThreads) void head_targets_kernel(Head h, const void* ids, bool wide, const void* teacher,
                                                                bool teacher16, float temperature, const uint16_t* x, float* loss,
                                                                uint16_t* dx) {
  const int lane = threadIdx.x % kWave;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / kWave) + threadIdx.x / kWave;
  if (t >= h.n) return;
  constexpr int kSlots = kMaxTop / kWave;
  int row[kSlots];
  float z[kSlots], top = -INFINITY;
  const int k = max(h.top, 1);
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int s = i * kWave + lane;
    row[i] = kNone;
    z[i] = -INFINITY;
    if (s < k) {
      const int64_t at = t * k + s;
      const int64_t v = wide ? static_cast<const int64_t*>(ids)[at] : static_cast<const int32_t*>(ids)[at];
      if (v >= 0 && v < h.rows) {
        row[i] = static_cast<int>(v);
        z[i] = !teacher ? 0.0f : teacher16 ? In<true>::elem(teacher, at) : In<false>::elem(teacher, at);
      }
    }
    top = fmaxf(top, z[i]);
  }
  bool some = false;   // a teacher's logit of -inf is no target, one of NaN is
#pragma unroll
  for (int i = 0; i < kSlots; ++i) some |= row[i] != kNone && !(z[i] == -INFINITY);
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
  some = __any(some);
  float sum = 0.0f, ent = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    z[i] = row[i] != kNone && some ? expf((z[i] - top) / temperature) : 0.0f;
    sum += z[i];
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    z[i] = some ? z[i] / sum : 0.0f;
    if (!(z[i] == 0.0f)) ent += z[i] * logf(z[i]);
  }
  int rank[kSlots] = {};   // by row, equal ones by place
#pragma unroll
  for (int r = 0; r < kSlots; ++r)
    for (int l = 0; l < kWave && r * kWave + l < k; ++l) {
      const int other = __builtin_amdgcn_readlane(row[r], l);
#pragma unroll
      for (int i = 0; i < kSlots; ++i) rank[i] += other < row[i] || (other == row[i] && r * kWave + l < i * kWave + lane);
    }
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (i * kWave + lane < k) {
      h.idx[t * k + rank[i]] = row[i];
      h.q[t * k + rank[i]] = z[i];
    }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) ent += __shfl_xor(ent, o, kWave);
  float most = 0.0f;
  if constexpr (GRAD) {
    if (some) {
      const uint16_t* from = x + t * h.cols;
      if (h.cols % 8 == 0) {
        for (int c = lane * 8; c < h.cols; c += kWave * 8) {
          float v[8];
          In<true>::widen(*reinterpret_cast<const u32x4*>(from + c), v);
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fabsf(v[e]) <= FLT_MAX ? fmaxf(most, fabsf(v[e])) : most;
        }
      } else {
        for (int c = lane; c < h.cols; c += kWave) {
          const float v = fabsf(In<true>::elem(from, c));
          most = v <= FLT_MAX ? fmaxf(most, v) : most;
        }
      }
#pragma unroll
      for (int o = kWave / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, kWave));
    } else if (h.cols % 8 == 0) {
      for (int c = lane * 8; c < h.cols; c += kWave * 8) *reinterpret_cast<u32x4*>(dx + t * h.cols + c) = u32x4{};
    } else {
      for (int c = lane; c < h.cols; c += kWave) dx[t * h.cols + c] = 0;
    }
  }
  if (lane == 0) {
    h.keep[t] = some;
    h.ent[t] = ent;
    h.xmax[t] = most;
    if (!some) loss[t] = 0.0f;
  }
}

// Parts of the contraction of dx: none, or as many as fill one to four rounds of
// the 256 CUs, whichever makes the launch shortest, counted in stages, with six
// for a part's ends; at least four stages a part. At most kMaxSlabs workgroups
// have a part each, which bounds the slabs.
constexpr int kMaxSlabs = 1024;
__host__ __device__ inline int dx_splits(int tiles, int ksteps) {
  if (tiles <= 0) return 1;
  int best = 1, least = (tiles + 255) / 256 * (ksteps + 6);
  for (int round = 1; round <= kMaxSlabs / 256; ++round) {
    int s = 256 * round / tiles;
    s = s < ksteps / 4 ? s : ksteps / 4;
    if (s < 2) continue;
    const int cost = (s * tiles + 255) / 256 * ((ksteps + s - 1) / s + 6);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

// The tokens with a target, in their order, by one workgroup; the exponents
// that bound x and a; and the pieces.
constexpr int kKeepThreads = 1024;
__global__ __launch_bounds__(kKeepThreads) void head_keep_kernel(Head h, const float* weights, float factor, int n_pieces,
                                                                 int dx_tiles_m, int tile_n) {
  __shared__ int wave_sum[kKeepThreads / kWave];
  __shared__ float wave_x[kKeepThreads / kWave], wave_a[kKeepThreads / kWave];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  int base = 0;
  float most_x = 0.0f, most_a = 0.0f;
  for (int t0 = 0; t0 < h.n; t0 += kKeepThreads) {
    const int t = t0 + tid;
    const bool mine = t < h.n && h.keep[t];
    const uint64_t set = __ballot(mine);
    if (lane == 0) wave_sum[wave] = __popcll(set);
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < kKeepThreads / kWave; ++w) {
      before += w < wave ? wave_sum[w] : 0;
      all += wave_sum[w];
    }
    __syncthreads();
    base += all;
    if (mine) {
      h.kept[before + __popcll(set & ((1ull << lane) - 1))] = t;
      const float a = fabsf((weights ? weights[t] : 1.0f) * factor);
      if (a != 0.0f) most_x = fmaxf(most_x, h.xmax[t]);   // others have zeros as fp16
      if (a <= FLT_MAX) most_a = fmaxf(most_a, a);
    }
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) {
    most_x = fmaxf(most_x, __shfl_xor(most_x, o, kWave));
    most_a = fmaxf(most_a, __shfl_xor(most_a, o, kWave));
  }
  if (lane == 0) {
    wave_x[wave] = most_x;
    wave_a[wave] = most_a;
  }
  __syncthreads();
  for (int w = 0; w < kKeepThreads / kWave; ++w) {
    most_x = fmaxf(most_x, wave_x[w]);
    most_a = fmaxf(most_a, wave_a[w]);
  }
  if (tid == 0) {
    int ex = 0, ec = 0;
    frexpf(most_x, &ex);   // 0 for 0
    frexpf(most_a, &ec);
    *h.info = HeadInfo{base, ex, ec, 0};
  }
  for (int p = tid; p < n_pieces; p += kKeepThreads) {
    const int count = min(max(base - p * h.piece, 0), h.piece);
    h.pieces[p] = HeadPiece{count, dx_splits(dx_tiles_m * ((count + tile_n - 1) / tile_n), h.vp / kStep)};
  }
}

// x of the kept tokens beside each other, as bf16 and (GRAD) scaled as fp16,
// zeros in the padding of their columns and in the places up to the next
// multiple of kStep; and their targets. A token whose gradient has no weight
// has zeros as fp16, whatever x holds.
template <bool GRAD>
__global__ __launch_bounds__(kThreads) void head_gather_kernel(Head h, const uint16_t* x, const float* weights, float factor) {
  const int p = blockIdx.x, count = h.info->count;
  if (p >= (count + kStep - 1) / kStep * kStep) return;
  const bool live = p < count;
  const int64_t t = live ? h.kept[p] : 0;
  const float a = live ? (weights ? weights[t] : 1.0f) * factor : 0.0f;
  const int shift = 14 - h.info->ex;
  if (live) {
    const int k = max(h.top, 1);
    for (int s = threadIdx.x; s < k; s += kThreads) {
      h.pidx[static_cast<int64_t>(p) * k + s] = h.idx[t * k + s];
      h.pq[static_cast<int64_t>(p) * k + s] = h.q[t * k + s];
    }
    if (threadIdx.x == 0) {
      h.pent[p] = h.ent[t];
      h.a[p] = a;
    }
  }
  const bool vec = h.cols % 8 == 0;
  const int wide = GRAD ? (h.cols + kTileM - 1) / kTileM * kTileM : h.hp;
  for (int c = threadIdx.x * 8; c < wide; c += kThreads * 8) {
    float v[8] = {};
    u32x4 raw = {};
    if (live && vec) {
      if (c < h.cols) raw = *reinterpret_cast<const u32x4*>(x + t * h.cols + c);
    } else if (live) {
      uint32_t e16[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) e16[e] = c + e < h.cols ? x[t * h.cols + c + e] : 0u;
      raw = u32x4{e16[0] | e16[1] << 16, e16[2] | e16[3] << 16, e16[4] | e16[5] << 16, e16[6] | e16[7] << 16};
    }
    if (c < h.hp)
      *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(h.xb) + (static_cast<int64_t>(c / kStep) * h.npad + p) * kStep + c % kStep) = raw;
    if constexpr (GRAD) {
      In<true>::widen(raw, v);
      h8 y;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = a == 0.0f ? static_cast<_Float16>(0.0f) : static_cast<_Float16>(ldexpf(v[e], shift));
      *reinterpret_cast<h8*>(reinterpret_cast<_Float16*>(h.xh) + (static_cast<int64_t>(c / kTileM) * h.npad + p) * kTileM + c % kTileM) = y;
    }
  }
}

// The table with its rows padded, where their width is no multiple of kStep. Bound
// by memory: 76552 x 4184 in 235 us, 5.5 TB/s (two bytes a lane: 400).
__global__ __launch_bounds__(kThreads) void head_widen_kernel(const uint16_t* table, int rows, int cols, int hp, uint16_t* out) {
  const int per = hp / 8;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (u >= static_cast<int64_t>(rows) * per) return;
  const int64_t r = u / per;
  const int c = static_cast<int>(u - r * per) * 8;
  const uint16_t* from = table + r * cols + c;
  u32x4 v = {};
  if (c + 8 <= cols) {
    __builtin_memcpy(&v, from, 16);   // one load, aligned or not
  } else {
    uint32_t e16[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) e16[e] = c + e < cols ? from[e] : 0u;
    v = u32x4{e16[0] | e16[1] << 16, e16[2] | e16[3] << 16, e16[4] | e16[5] << 16, e16[6] | e16[7] << 16};
  }
  *reinterpret_cast<u32x4*>(out + r * hp + c) = v;
}

// ------------------------------------------------------------------ logits

// Exponentials are powers of two: 2^(l log2(e) - z), with maxima, log-sums and
// z in powers of two, so that the product is not rounded by itself.
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// Where the logit of row c (rows c to c | 3) and a place of the piece lies:
// blocks of 256 rows by 32 tokens, in them the order of the accumulators, so that
// a wave stores 1 KB at once (4096 tokens by 131072 rows of 4096: 3.70 ms; token
// after token, 32 bytes at once, 3.85).
__device__ __forceinline__ float* logit_at(const Head& h, int c, int place) {
  const int block = place / 32 * 32, row = c % kTileM;
  return h.logits + (static_cast<int64_t>(c / kTileM) * h.piece + block) * kTileM + row / 8 * 256 + (row / 4 % 2 * 32 + place - block) * 4 + row % 4;
}

// What is kept of one tile of the logits: for each token the largest and the
// sum of exponentials over the wave's rows, and the logits themselves, -inf
// behind the table's end (STORE), or those at its targets, which are sorted. A lane
// holds one token's logits, so the sums are its own and the other half wave's.
template <class T, bool STORE>
__device__ __forceinline__ void keep_logits(const Head& h, int piece, int count, const TileAt& at, float factor, HeadAcc<T>& acc) {
  const int tid = fresh_thread(), lane = tid % kWave, wave = tid / kWave, half = lane / 32;
  const int row = wave / T::WC * T::NI * 32, first = at.m * kTileM + row;   // the wave's first row, in the tile and of the table
  const bool inside = first + T::NI * 32 <= h.rows;
  // each token's first target that is no row ahead of the wave's
  const int k = STORE ? 0 : max(h.top, 1);
  int slot[T::NJ], to[T::NJ];
#pragma unroll
  for (int j = 0; j < T::NJ; ++j) {
    slot[j] = 0;
    to[j] = at.n * T::kN + (wave % T::WC * T::NJ + j) * 32 + lane % 32 < count ? k : 0;
  }
  for (int left = k; left > 0; left >>= 1) {
    int row_at[T::NJ];
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) {
      const int64_t mine = static_cast<int64_t>(piece) * h.piece + at.n * T::kN + (wave % T::WC * T::NJ + j) * 32 + lane % 32;
      row_at[j] = slot[j] < to[j] ? h.pidx[mine * k + (slot[j] + to[j]) / 2] : 0;
    }
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) {
      const int mid = (slot[j] + to[j]) / 2;
      if (slot[j] < to[j] && row_at[j] < first) slot[j] = mid + 1;
      else to[j] = mid;
    }
  }
#pragma unroll
  for (int j = 0; j < T::NJ; ++j) {
    const int place = at.n * T::kN + (wave % T::WC * T::NJ + j) * 32 + lane % 32;   // in the piece
    const bool live = place < count;
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc.v[i][j][e] *= factor;
    if (!inside) {
#pragma unroll
      for (int i = 0; i < T::NI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (first + i * 32 + e / 4 * 8 + half * 4 + e % 4 >= h.rows) acc.v[i][j][e] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, acc.v[i][j][e]);
    top = fmaxf(top, __shfl_xor(top, 32, kWave)) * kLog2e;
    const float base = top == -INFINITY ? 0.0f : top;   // only -inf and NaN: the sum says which
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) sum += exp2_of(__builtin_fmaf(acc.v[i][j][e], kLog2e, -base));
    sum += __shfl_xor(sum, 32, kWave);
    if (live && half == 0) h.stat[static_cast<int64_t>(first / (32 * T::NI)) * h.piece + place] = float2{top, sum};
    if constexpr (!STORE) {
      const int64_t mine = static_cast<int64_t>(piece) * h.piece + place;
      if (live)
        for (int t = slot[j]; t < k; ++t) {
          const int hit = h.pidx[mine * k + t] - first;
          if (hit >= T::NI * 32) break;
          if (hit / 4 % 2 != half) continue;
          float l = 0.0f;
#pragma unroll
          for (int i = 0; i < T::NI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) l = hit == i * 32 + e / 4 * 8 + half * 4 + e % 4 ? acc.v[i][j][e] : l;
          h.picked[mine * k + t] = l;
        }
    }
    if constexpr (STORE) {
      if (live) {
        float* out = logit_at(h, first + half * 4, place);
#pragma unroll
        for (int i = 0; i < T::NI; ++i)
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<f32x4*>(out + i * 1024 + e * 64) =
                f32x4{acc.v[i][j][e], acc.v[i][j][e + 1], acc.v[i][j][e + 2], acc.v[i][j][e + 3]};
      }
    }
  }
}

// Tiles of the logits of a piece, 256 rows of the table by BN tokens; one
// workgroup a CU, which takes tile after tile and loads the next one while it keeps
// this one. Bound by the matrix cores: 4096 x 131072 x 4096 in 3.73 ms with the
// logits stored and 3.65 without, 1180 and 1205 TFLOP/s; by memory for up to
// 64 tokens (48 x 131072 x 4096: 178 us, 6.0 TB/s of the table).
template <class T, bool STORE>
__global__ __launch_bounds__(T::kThreads) void head_logits_kernel(Head h, int piece, float factor) {
  constexpr int BN = T::kN;
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  const int count = h.pieces[piece].count, m_tiles = h.vp / kTileM, n_tiles = (count + BN - 1) / BN;
  Items items(m_tiles * n_tiles);
  if (items.now >= items.end) return;
  const int64_t x_step = static_cast<int64_t>(h.npad) * (kStep * 2);
  Contract<T, false, false, false, false, false> product(lds);
  auto begin = [&](const TileAt& at) {
    const int64_t from = static_cast<int64_t>(at.m * kTileM) * h.pitch;
    const int64_t x_from = (static_cast<int64_t>(piece) * h.piece + at.n * BN) * (kStep * 2);
    product.begin({h.table + from, h.table_bytes - from, h.pitch, h.rows - at.m * kTileM, kStep * 2},
                  {h.xb + x_from, h.hp / kStep * x_step - x_from, kStep * 2, BN, x_step}, h.hp / kStep, false, 0);
  };
  TileAt at = tile_at(items.now, n_tiles, m_tiles, false);
  begin(at);
  for (bool ahead = false;; ahead = true) {
    HeadAcc<T> acc;
    product.run(acc, ahead);
    const TileAt done = at;
    items.now += items.stride;
    const bool more = items.now < items.end;
    if (more) begin(at = tile_at(items.now, n_tiles, m_tiles, false));
    keep_logits<T, STORE>(h, piece, count, done, factor, acc);
    if (!more) return;
  }
}

// Log-sum-exp and loss of TOKENS tokens, and (STORED) the logits at their targets
// out of the stored ones. The largest logit and the logarithm stay two numbers, and
// a logit's distance is taken from the first ahead of the second: added up in one
// fp32 number, a loss of 1e-6 at logits of 100 is off by up to 9e-6 and negative at
// times (so by 1e-6 at most, and never). A token's numbers lie a piece apart, so
// eight neighbours share what a load brings; few tokens take a workgroup each. Bound
// by latency: 15 us for 4096 tokens with 1024 numbers each (34 MB).
template <int TOKENS, bool STORED>
__global__ __launch_bounds__(kThreads) void head_loss_kernel(Head h, int piece, int stats, float factor, float* loss) {
  constexpr int kParts = kThreads / TOKENS;
  __shared__ float tops[TOKENS][kParts + 1], sums[TOKENS][kParts + 1];
  const int tok = threadIdx.x % TOKENS, part = threadIdx.x / TOKENS;
  const int place = blockIdx.x * TOKENS + tok, count = h.pieces[piece].count;
  const bool live = place < count;
  const int64_t mine = static_cast<int64_t>(piece) * h.piece + place;
  float top = -INFINITY, sum = 0.0f;
  bool broken = false;
  auto add = [&](float t, float s) {
    const float both = fmaxf(top, t), base = both == -INFINITY ? 0.0f : both;
    broken |= !(s >= 0.0f);
    sum = sum * exp2_of(top - base) + s * exp2_of(t - base);
    top = both;
  };
  if (live)
#pragma unroll 4
    for (int i = part; i < stats; i += kParts) {
      const float2 s = h.stat[static_cast<int64_t>(i) * h.piece + place];
      add(s.x, s.y);
    }
  for (int width = kParts; width > 1; width /= 2) {   // the upper half joins the lower one
    __syncthreads();
    if (part >= width / 2 && part < width) {
      tops[tok][part] = top;
      sums[tok][part] = broken ? NAN : sum;
    }
    __syncthreads();
    if (part < width / 2) add(tops[tok][part + width / 2], sums[tok][part + width / 2]);
  }
  if (part == 0) {
    tops[tok][kParts] = top;
    sums[tok][kParts] = broken ? NAN : log2f(sum);
  }
  __syncthreads();
  const float2 z = {tops[tok][kParts], sums[tok][kParts]};
  float l = 0.0f;
  const int k = max(h.top, 1);
  if (live)
    for (int s = part; s < k; s += kParts) {
      const int64_t at = mine * k + s;
      const int c = h.pidx[at];
      if (c == kNone) continue;
      float y;
      if constexpr (STORED) h.picked[at] = y = *logit_at(h, c, place);
      else y = h.picked[at];
      const float q = h.pq[at];
      const float far = z.y - __builtin_fmaf(y, kLog2e, -z.x);   // -log2 p, under 0 by rounding alone
      if (!(q == 0.0f)) l += q * (far < 0.0f ? 0.0f : far * kLn2);
    }
  sums[tok][part] = l;
  __syncthreads();
  if (part || !live) return;
  l = 0.0f;
  for (int i = 0; i < min(k, kParts); ++i) l += sums[tok][i];
  h.lse[mine] = z;
  loss[h.kept[mine]] = factor * (h.pent[mine] + l);
}

// ------------------------------------------------------------------ gradients

// A product that is split: both parts must be of one value, where the compiler
// otherwise multiplies a second time with a single rounding to fp16, which ends on
// the other side of a tie now and then.
__device__ __forceinline__ float one_value(float x) {
  asm("" : "+v"(x));
  return x;
}

// Bound by memory: 4096 tokens by 131072 rows in 0.85 ms, 5.1 TB/s.
// d = p - q of a block of 32 tokens and 256 columns: bf16 for dx, and times the
// token's share of the gradient, scaled, in fp16 parts for dW, where the logits
// lay, in rows of 256 columns a token: 64 logits give way to 64 values of each
// part. The whole block is read ahead of the first write.
constexpr int kDeltaTokens = 32;
template <bool TWO>
__global__ __launch_bounds__(kThreads) void head_delta_kernel(Head h, int piece) {
  const int count = h.pieces[piece].count, places = (count + kStep - 1) / kStep * kStep;
  const int t0 = blockIdx.x * kDeltaTokens, c0 = blockIdx.y * kTileM;
  if (t0 >= places) return;
  const int64_t first = static_cast<int64_t>(piece) * h.piece;
  const int up = 15 - h.info->ec;
  auto part = [&](int place, int c) {
    return reinterpret_cast<_Float16*>(h.logits + (static_cast<int64_t>(c / kTileM) * h.piece + place) * kTileM + c % kTileM / kPart * kPart) + c % kPart;
  };
  auto d16 = [&](int place, int c) { return h.d + (static_cast<int64_t>(c / kStep) * h.piece + place) * kStep + c % kStep; };
  constexpr int kUnits = kDeltaTokens * kTileM / 8 / kThreads;   // of 8 columns, 64 columns of 8 tokens a wave
  static_assert(kDeltaTokens == kThreads / kWave * 8 && kUnits == kTileM / kPart, "a wave has its tokens");
  const int lane = threadIdx.x % kWave, place = t0 + threadIdx.x / 8, c1 = c0 + lane % 8 * 8;
  const float a = place < count ? h.a[first + place] : 0.0f;
  const float2 z = a != 0.0f ? h.lse[first + place] : float2{};
  const float g = ldexpf(a, up);
  f32x4 l[kUnits][2] = {};
  if (a != 0.0f) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      l[u][0] = *reinterpret_cast<const f32x4*>(logit_at(h, c1 + u * kPart, place));
      l[u][1] = *reinterpret_cast<const f32x4*>(logit_at(h, c1 + u * kPart + 4, place));
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int c = c1 + u * kPart;
    u32x4 out = {};
    h8 hi = {}, lo = {};
    if (a != 0.0f) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = exp2_of(__builtin_fmaf(l[u][e / 4][e % 4], kLog2e, -z.x) - z.y);
        const float y = one_value(p[e] * g);
        hi[e] = static_cast<_Float16>(y);
        lo[e] = static_cast<_Float16>(y - static_cast<float>(hi[e]));
      }
      out = u32x4{bf16_pair(p[0], p[1]), bf16_pair(p[2], p[3]), bf16_pair(p[4], p[5]), bf16_pair(p[6], p[7])};
    }
    *reinterpret_cast<u32x4*>(d16(place, c)) = out;
    *reinterpret_cast<h8*>(part(place, c)) = hi;
    if constexpr (TWO) *reinterpret_cast<h8*>(part(place, c) + kPart) = lo;
  }
  __syncthreads();   // the targets' columns again, with their share; the first of equal rows has all of it
  const int k = max(h.top, 1);
  for (int i = threadIdx.x; i < k * kDeltaTokens; i += kThreads) {
    const int to = t0 + i / k, slot = i % k;
    if (to >= count) continue;
    const int64_t mine = first + to, at = mine * k;
    const int c = h.pidx[at + slot];
    const float a = h.a[mine];
    if (c < c0 || c >= c0 + kTileM || a == 0.0f) continue;
    if (slot && h.pidx[at + slot - 1] == c) {
      h.rest[at + slot] = 0.0f;
      continue;
    }
    float q = 0.0f;
    for (int s = slot; s < k && h.pidx[at + s] == c; ++s) q += h.pq[at + s];
    const float2 z = h.lse[mine];
    const float p = exp2_of(__builtin_fmaf(h.picked[at + slot], kLog2e, -z.x) - z.y) - q, y = one_value(p * ldexpf(a, up));
    const uint32_t rounded = bf16_rne(p);
    *d16(to, c) = static_cast<uint16_t>(rounded);
    h.rest[at + slot] = p - __builtin_bit_cast(float, rounded << 16);
    const _Float16 hi = static_cast<_Float16>(y);
    *part(to, c) = hi;
    if constexpr (TWO) part(to, c)[kPart] = static_cast<_Float16>(y - static_cast<float>(hi));
  }
}

// What the rounding of d to bf16 leaves of a token's targets, where most of d is,
// times their rows of the table, for dx to add in fp32: a workgroup a token. The
// other rows' roundings are many and small and of both signs. With it dx's error is
// that of its own rounding (0.0017 of it; without 0.0018 for labels and 0.0023 to
// 0.0025 for a teacher's 7 to 64 places), for 1 to 2% of the call's time.
__global__ __launch_bounds__(kThreads) void head_rest_kernel(Head h, int piece) {
  const int place = blockIdx.x;
  if (place >= h.pieces[piece].count) return;
  const int k = max(h.top, 1);
  const int64_t mine = static_cast<int64_t>(piece) * h.piece + place;
  if (h.a[mine] == 0.0f) return;   // nor does dx read it
  for (int c = threadIdx.x * 8; c < h.hp; c += kThreads * 8) {
    float sum[8] = {};
    for (int s = 0; s < k; ++s) {
      const int row = h.pidx[mine * k + s];
      if (row == kNone) break;
      const float r = h.rest[mine * k + s];
      if (r == 0.0f) continue;
      float w[8];
      In<true>::widen(*reinterpret_cast<const u32x4*>(h.table + static_cast<int64_t>(row) * h.pitch + c * 2), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(r, w[e], sum[e]);
    }
    f32x4* out = reinterpret_cast<f32x4*>(h.fix + static_cast<int64_t>(place) * h.hp + c);
    out[0] = f32x4{sum[0], sum[1], sum[2], sum[3]};
    out[1] = f32x4{sum[4], sum[5], sum[6], sum[7]};
  }
}

// dx of a piece: 256 columns by BN tokens, one part of the contraction over the
// table's rows (see dx_splits). Sums go to the part's slab, in the registers'
// order. Bound by the matrix cores: 4096 x 131072 x 4096 in 3.0 to 3.2 ms; by
// memory for few tokens (48 x 131072 x 1024: 48 us, 5.9 TB/s).
template <int BN>
__global__ __launch_bounds__(DxTile<BN>::kThreads) void head_dx_kernel(Head h, int piece) {
  using T = DxTile<BN>;
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  const HeadPiece info = h.pieces[piece];
  const int m_tiles = (h.cols + kTileM - 1) / kTileM, n_tiles = (info.count + BN - 1) / BN, tiles = m_tiles * n_tiles;
  const Items items(tiles * info.splits);
  const int o = items.now;
  if (o >= items.end) return;
  const int split = o / tiles;
  const TileAt at = tile_at(o - split * tiles, m_tiles, n_tiles, true);
  const int ksteps = h.vp / kStep;
  const int k0 = static_cast<int>(static_cast<int64_t>(ksteps) * split / info.splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(ksteps) * (split + 1) / info.splits);
  // stages behind the table's last row repeat it; d is zero there
  const int row = min(k0 * kStep, h.rows - 1);
  const int64_t from = static_cast<int64_t>(row) * h.pitch + at.m * (kTileM * 2);
  const int64_t d_step = static_cast<int64_t>(h.piece) * (kStep * 2), d_from = k0 * d_step + at.n * (BN * kStep * 2);
  HeadAcc<T> acc;
  Contract<T, false, true, false, true, false> product(lds);
  product.begin({h.table + from, h.table_bytes - from, h.pitch, h.rows - row, 0},
                {reinterpret_cast<const char*>(h.d) + d_from, ksteps * d_step - d_from, kStep * 2, BN, d_step}, k1 - k0, false, 0);
  product.run(acc, false);
  char* out = h.slabs + static_cast<int64_t>(o) * (kTileM * BN * 4) + fresh_thread() * 16;
#pragma unroll
  for (int i = 0; i < T::NI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<f32x4*>(out + ((i * T::NJ + j) * 4 + e / 4) * (T::kThreads * 16)) =
            f32x4{acc.v[i][j][e], acc.v[i][j][e + 1], acc.v[i][j][e + 2], acc.v[i][j][e + 3]};
}

// dx of one 32-column block of a tile for each of its waves: the parts added in
// their order, times a, rounded to bf16, to the tokens' own rows.
template <int BN>
__global__ __launch_bounds__(DxTile<BN>::kThreads) void head_dx_sum_kernel(Head h, int piece, uint16_t* dx) {
  using T = DxTile<BN>;
  constexpr int kBlocks = T::NI * T::NJ * 4;
  const HeadPiece info = h.pieces[piece];
  const int m_tiles = (h.cols + kTileM - 1) / kTileM, n_tiles = (info.count + BN - 1) / BN, tiles = m_tiles * n_tiles;
  const int tile = blockIdx.x / kBlocks, block = blockIdx.x % kBlocks;
  if (tile >= tiles) return;
  const TileAt at = tile_at(tile, m_tiles, n_tiles, true);
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int i = block / 4 / T::NJ, j = block / 4 % T::NJ, e4 = block % 4;
  const int place = at.n * BN + (wave % T::WC * T::NJ + j) * 32 + lane % 32;
  const int c = at.m * kTileM + (wave / T::WC * T::NI + i) * 32 + e4 * 8 + lane / 32 * 4;
  if (place >= info.count || c >= h.cols) return;
  const char* from = h.slabs + static_cast<int64_t>(tile) * (kTileM * BN * 4) + block * (T::kThreads * 16) + tid * 16;
  f32x4 sum = {};
#pragma unroll 4
  for (int s = 0; s < info.splits; ++s) sum += *reinterpret_cast<const f32x4*>(from + static_cast<int64_t>(s) * tiles * (kTileM * BN * 4));
  const int64_t mine = static_cast<int64_t>(piece) * h.piece + place;
  const float a = h.a[mine];
  if (a != 0.0f) sum += *reinterpret_cast<const f32x4*>(h.fix + static_cast<int64_t>(place) * h.hp + c);
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = bf16_rne(a == 0.0f ? 0.0f : sum[e] * a);
  uint16_t* out = dx + static_cast<int64_t>(h.kept[mine]) * h.cols + c;
  if (h.cols % 4 == 0) {
    *reinterpret_cast<u32x2*>(out) = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < h.cols) out[e] = static_cast<uint16_t>(b[e]);
  }
}

// How a value of dW is finished: out <- [in +] sigma * 2^up * x. The factor is
// two, either of which fp32 holds; adding 0 leaves no -0.0.
template <bool OUT16>
struct Finish {
  const float* in;
  void* out;
  float f0, f1;

  __device__ __forceinline__ float value(float x, float before) const { return __builtin_fmaf(x * f0, f1, before + 0.0f); }
  __device__ __forceinline__ void one(int64_t at, float x) const {
    const float y = value(x, in ? in[at] : 0.0f);
    if constexpr (OUT16) static_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(bf16_rne(y));
    else static_cast<float*>(out)[at] = y;
  }
  __device__ __forceinline__ f32x4 before(int64_t at) const { return in ? *reinterpret_cast<const f32x4*>(in + at) : f32x4{}; }
  __device__ __forceinline__ void four(int64_t at, const f32x4& x, const f32x4& b) const {
    const f32x4 y = {value(x[0], b[0]), value(x[1], b[1]), value(x[2], b[2]), value(x[3], b[3])};
    if constexpr (OUT16) *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + at) = u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
    else *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = y;
  }
};

// A tile of dW where rows are 16-byte aligned (fp32): every lane has four
// neighbours of a row, and four stores of a wave fill 128 bytes of 32 rows.
template <bool OUT16>
__device__ __forceinline__ void keep_dw(const Head& h, const TileAt& at, const Finish<OUT16>& f, const HeadAcc<DwTile>& acc) {
  using T = DwTile;
  const int tid = fresh_thread(), lane = tid % kWave, wave = tid / kWave;
#pragma unroll
  for (int j = 0; j < T::NJ; ++j) {
    const int v = at.n * T::kN + (wave % T::WC * T::NJ + j) * 32 + lane % 32;
    if (v >= h.rows) continue;
    const int c = at.m * kTileM + wave / T::WC * T::NI * 32 + lane / 32 * 4;
    const int64_t to = static_cast<int64_t>(v) * h.cols + c;
#pragma unroll
    for (int i = 0; i < T::NI; ++i) {
      f32x4 b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = c + i * 32 + e * 8 < h.cols ? f.before(to + i * 32 + e * 8) : f32x4{};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x16& x = acc.v[i][j];
        if (c + i * 32 + e * 8 < h.cols) f.four(to + i * 32 + e * 8, f32x4{x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]}, b[e]);
      }
    }
  }
}

// The same for rows of any alignment: half of the tile's rows at a time go
// through LDS, 1 KiB each, and a wave reads and writes whole rows. Piece c of row
// r lies at place c ^ (r % 32). 32001 x 1001 and 517 tokens: 187 us, single
// elements out of the registers 405. Where rows are aligned it is no faster
// (131072 x 4096 and 4096 tokens: 7.13 ms against 7.03, 512 tokens 258 us against
// 250), so these have keep_dw.
template <bool OUT16>
__device__ __forceinline__ void keep_dw_odd(const Head& h, const TileAt& at, const Finish<OUT16>& f, const HeadAcc<DwTile>& acc, char* lds) {
  using T = DwTile;
  constexpr int kHalf = T::NJ / 2, kRows = T::kN / 2;
  static_assert(kRows * kTileM * 4 <= T::kLds, "half a tile");
  const int tid = fresh_thread(), lane = tid % kWave, wave = tid / kWave;
  const int width = min(h.cols - at.m * kTileM, kTileM);
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if (pass) barrier();
#pragma unroll
    for (int jj = 0; jj < kHalf; ++jj)
#pragma unroll
      for (int i = 0; i < T::NI; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const f32x16& x = acc.v[i][pass * kHalf + jj];
          const int r = (wave % T::WC * kHalf + jj) * 32 + lane % 32;
          const int c = (wave / T::WC * T::NI + i) * 8 + e / 2 + lane / 32;
          *reinterpret_cast<f32x4*>(lds + r * (kTileM * 4) + (c ^ r % 32) * 16) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
        }
    wait<63, true>();
    barrier();
    for (int r = wave * (kRows / T::kWaves); r < (wave + 1) * (kRows / T::kWaves); ++r) {
      const int v = at.n * T::kN + (r / 32 / kHalf * T::NJ + pass * kHalf + r / 32 % kHalf) * 32 + r % 32;
      if (v >= h.rows) continue;
      const int64_t to = static_cast<int64_t>(v) * h.cols + at.m * kTileM;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int c = t * kWave + lane;
        if (c < width) f.one(to + c, *reinterpret_cast<const float*>(lds + r * (kTileM * 4) + (c / 4 ^ r % 32) * 16 + c % 4 * 4));
      }
    }
  }
  barrier();
}

// Tiles of dW of a piece, 256 columns by 256 rows of the table; one workgroup a
// CU, with tile after tile (512 tokens, 131072 x 1024: 259 us, one tile a workgroup
// 285). Bound by the matrix cores: 1250 TFLOP/s with
// two parts, 1170 with one; for few tokens by the tiles' stores, one CU with one
// tile at a time. The tokens of a piece are not split: a small table has few tiles,
// whose CUs walk all of them (the whole call on 1000 x 64 with 2048, 8192, 16384
// tokens, fp32: 134, 354, 698 us).
template <bool TWO, bool OUT16>
__global__ __launch_bounds__(DwTile::kThreads) void head_dw_kernel(Head h, int piece, float sigma, const float* in, void* out) {
  using T = DwTile;
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  const HeadInfo info = *h.info;
  const int count = h.pieces[piece].count, depth = (count + kStep - 1) / kStep * kStep;
  if (count == 0 && in == out) return;   // nothing to add
  const int m_tiles = (h.cols + kTileM - 1) / kTileM, n_tiles = h.vp / T::kN;
  Items items(m_tiles * n_tiles);
  if (items.now >= items.end) return;
  const int up = info.ec + info.ex - 29;
  const Finish<OUT16> finish = {in, out, __builtin_ldexpf(1.0f, up / 2), __builtin_ldexpf(sigma, up - up / 2)};
  constexpr int kRow = kTileM * 2, kRowD = T::kN * 4, kLow = TWO ? kPart * 2 : 0;
  Contract<T, true, true, true, false, true> product(lds);
  auto begin = [&](const TileAt& at) {
    const int64_t x_from = (static_cast<int64_t>(at.m) * h.npad + static_cast<int64_t>(piece) * h.piece) * kRow;
    const int64_t d_from = static_cast<int64_t>(at.n) * h.piece * kRowD + kLow;
    product.begin({h.xh + x_from, static_cast<int64_t>(m_tiles) * h.npad * kRow - x_from, kRow, depth, 0},
                  {reinterpret_cast<const char*>(h.logits) + d_from, static_cast<int64_t>(n_tiles) * h.piece * kRowD - d_from, kRowD, depth, 0},
                  (TWO ? 2 : 1) * depth / kStep, TWO, -kLow);
  };
  const bool odd = h.cols % 4 != 0;
  TileAt at = tile_at(items.now, m_tiles, n_tiles, true);
  begin(at);
  for (bool ahead = false;; ahead = true) {
    HeadAcc<T> acc;
    product.run(acc, ahead);
    const TileAt done = at;
    items.now += items.stride;
    const bool more = items.now < items.end;
    if (more) at = tile_at(items.now, m_tiles, n_tiles, true);
    if (odd) {
      keep_dw_odd(h, done, finish, acc, lds);
      if (more) begin(at);
    } else {
      if (more) begin(at);
      keep_dw(h, done, finish, acc);
    }
    if (!more) return;
  }
}

// ------------------------------------------------------------------ host

constexpr int64_t kHeadMaxTokens = int64_t(1) << 20, kHeadMaxRows = int64_t(1) << 21, kHeadMaxCols = int64_t(1) << 16;
constexpr int64_t kHeadMaxElems = int64_t(1) << 33;
// Tokens of a piece, unless the call says another number (16384 tokens of 131072 x
// 4096, fp32 gradients: 57.7 ms; 59.6 with 4096, which halves the workspace).
constexpr int64_t kPieceTokens = 8192;
constexpr int64_t kPieceMax = 65536;
// Up to here a workgroup takes one token's loss, above it eight (131072 rows: 100
// tokens 8.7 us with one, 16.0 with eight; 200 7.7 and 11.1; 512 9.9 and 7.8; 1024
// 15.8 and 8.8).
constexpr int64_t kFewTokens = 256;
constexpr int64_t kCus = 256;   // workgroups of a product: one a CU, each with tile after tile

int64_t up_to(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// A call's sizes, its workspace laid out, and how it is launched.
struct HeadShape {
  int64_t n = 0, npad = 0, rows = 0, cols = 0, vp = 0, hp = 0, top = 0, piece = 0, n_pieces = 0;
  int tile_n = 256;            // tokens of a tile
  int64_t dx_groups = 0;       // workgroups of the dx product
  bool grad = false, widen = false, stored = false, sums = false;   // sums: dW adds up in the workspace
  int64_t info, pieces, keep, xmax, ent, idx, q, kept, pent, a, lse, pidx, pq, picked, xb, xh, stat, logits, d, slabs, rest, fix, table, acc;
  int64_t bytes = 0;
};

int head_shape(const rs_plan* p, int64_t tensor, int64_t n, int64_t top, bool grad, int32_t packed_dt, int64_t piece, const char* who,
               HeadShape* s) {
  if (tensor < 0 || tensor >= p->n) return fail(RS_EINVAL, std::string(who) + ": no such tensor");
  const Tensor& t = p->t[tensor];
  if (t.kind == RS_TILEMAJOR) return fail(RS_EINVAL, std::string(who) + ": a TILEMAJOR tensor has no contiguous rows");
  if (n < 0 || top < 0 || top > kMaxTop || piece < 0 || piece % 256 || piece > kPieceMax)
    return fail(RS_EINVAL, std::string(who) + ": tokens >= 0, 0 to 256 top logits, pieces of a multiple of 256 tokens up to 65536 (or 0)");
  if (n > kHeadMaxTokens || t.rows > kHeadMaxRows || t.cols > kHeadMaxCols || t.n > kHeadMaxElems || n * t.cols > kHeadMaxElems ||
      n * std::max<int64_t>(top, 1) > (int64_t(1) << 28))
    return fail(RS_ERANGE, std::string(who) + ": at most 2^20 tokens, 2^21 rows, 2^16 columns, table and tokens * columns at most 2^33 "
                               "elements, tokens * top at most 2^28");
  s->n = n;
  s->rows = t.rows;
  s->cols = t.cols;
  s->top = top;
  s->grad = grad;
  s->npad = up_to(n, 256);
  s->vp = up_to(t.rows, kTileM);
  s->hp = up_to(t.cols, kStep);
  s->widen = s->hp != t.cols;
  // pieces of equal size, of at most the tokens asked for; the workspace has room
  // for these, so that one for more tokens serves fewer
  const int64_t most = std::min(s->npad, piece ? piece : kPieceTokens);
  s->n_pieces = most ? (s->npad + most - 1) / most : 0;
  s->piece = s->n_pieces ? up_to((s->npad + s->n_pieces - 1) / s->n_pieces, 256) : 256;
  // tokens of a tile of the logits and dx (131072 x 1024: 48 tokens 82 + 48 us with
  // 64, 84 + 54 with 128, 104 + 77 with 256; 100 tokens 84 + 59 with 128, 105 + 82
  // with 256)
  s->tile_n = n <= 64 ? 64 : n <= 128 ? 128 : 256;
  // the logits at the targets: out of the stored logits where these are stored
  // anyway, or where a wave's rows would hold several of a token's targets; else
  // out of the registers
  s->stored = grad || t.rows < 256 * top;
  s->sums = grad && packed_dt == RS_BF16 && s->n_pieces > 1;
  const int64_t k = std::max<int64_t>(top, 1), dx_m = (t.cols + kTileM - 1) / kTileM;
  for (int64_t tt = 1; tt <= (std::min(most, n) + s->tile_n - 1) / s->tile_n; ++tt)
    s->dx_groups = std::max(s->dx_groups, dx_m * tt * dx_splits(static_cast<int>(dx_m * tt), static_cast<int>(s->vp / kStep)));
  int64_t at = 0;
  auto room = [&](int64_t bytes) {
    const int64_t here = at;
    at += up_to(bytes, 256);
    return here;
  };
  s->info = room(sizeof(HeadInfo));
  s->pieces = room(s->n_pieces * sizeof(HeadPiece));
  s->keep = room(n * 4);
  s->xmax = room(n * 4);
  s->ent = room(n * 4);
  s->idx = room(n * k * 4);
  s->q = room(n * k * 4);
  s->kept = room(s->npad * 4);
  s->pent = room(s->npad * 4);
  s->a = room(s->npad * 4);
  s->lse = room(s->npad * 8);
  s->pidx = room(s->npad * k * 4);
  s->pq = room(s->npad * k * 4);
  s->picked = room(s->npad * k * 4);
  s->xb = room(s->npad * s->hp * 2);
  s->stat = room(most * (s->vp / 64) * 8);
  s->table = room(s->widen ? s->rows * s->hp * 2 : 0);
  s->xh = room(grad ? s->npad * up_to(s->cols, kTileM) * 2 : 0);
  s->logits = room(s->stored ? most * s->vp * 4 : 0);
  s->d = room(grad ? most * s->vp * 2 : 0);
  s->rest = room(grad ? s->npad * k * 4 : 0);
  s->fix = room(grad ? most * s->hp * 4 : 0);
  s->slabs = room(grad ? s->dx_groups * kTileM * s->tile_n * 4 : 0);
  s->acc = room(s->sums ? s->rows * s->cols * 4 : 0);
  s->bytes = n ? at : 0;
  return RS_OK;
}

// What the four calls have in common.
struct HeadArgs {
  int64_t tensor;
  const void *gathered, *x;
  int64_t n;
  const void* ids;
  int32_t id_bytes;
  const void* teacher;    // null: ids are labels
  int32_t teacher_dt;
  int64_t top;
  float temperature, scale;
  float* loss;
  const float* weights;
  void* dx;
  const float* prev;
  void* packed;
  int32_t packed_dt, scale_mode;
  float grad_scale;
  int64_t piece;
  void* work;
  int64_t work_bytes;
};

template <int BN>
void launch_head(const HeadShape& s, const Head& h, const HeadArgs& a, float sigma, bool grad, float factor, hipStream_t q) {
  const float c = a.scale / a.temperature, f = a.temperature * a.temperature;
  for (int64_t i = 0; i < s.n_pieces; ++i) {
    const int piece = static_cast<int>(i);
    const int64_t tokens = std::min(s.piece, s.n - i * s.piece);
    const int64_t n_tiles = (tokens + BN - 1) / BN, m_tiles = s.vp / kTileM;
    const dim3 tiles(static_cast<unsigned>(std::min<int64_t>(up_to(m_tiles * n_tiles, 8), kCus)));
    auto logits = [&](auto tile) {
      using T = decltype(tile);
      static_assert(T::NI == HeadTile<BN>::NI, "rows of the statistics");
      if (s.stored) hipLaunchKernelGGL((head_logits_kernel<T, true>), tiles, dim3(T::kThreads), 0, q, h, piece, c);
      else hipLaunchKernelGGL((head_logits_kernel<T, false>), tiles, dim3(T::kThreads), 0, q, h, piece, c);
    };
    if (s.cols <= kShortCols) logits(HeadTile<BN>());
    else logits(DxTile<BN>());
    const int stats = static_cast<int>(s.vp / (32 * HeadTile<BN>::NI));
    const dim3 few(static_cast<unsigned>(tokens)), many(static_cast<unsigned>((tokens + 7) / 8));
    if (tokens <= kFewTokens && s.stored)
      hipLaunchKernelGGL((head_loss_kernel<1, true>), few, dim3(kThreads), 0, q, h, piece, stats, f, a.loss);
    else if (tokens <= kFewTokens)
      hipLaunchKernelGGL((head_loss_kernel<1, false>), few, dim3(kThreads), 0, q, h, piece, stats, f, a.loss);
    else if (s.stored)
      hipLaunchKernelGGL((head_loss_kernel<8, true>), many, dim3(kThreads), 0, q, h, piece, stats, f, a.loss);
    else
      hipLaunchKernelGGL((head_loss_kernel<8, false>), many, dim3(kThreads), 0, q, h, piece, stats, f, a.loss);
    if (!grad) continue;
    const bool two = a.packed_dt == RS_F32;
    const dim3 delta(static_cast<unsigned>(up_to(tokens, kStep) / kDeltaTokens), static_cast<unsigned>(s.vp / kTileM));
    if (two) hipLaunchKernelGGL(head_delta_kernel<true>, delta, dim3(kThreads), 0, q, h, piece);
    else hipLaunchKernelGGL(head_delta_kernel<false>, delta, dim3(kThreads), 0, q, h, piece);
    const int64_t dx_m = (s.cols + kTileM - 1) / kTileM;
    const dim3 dx_threads(DxTile<BN>::kThreads);
    hipLaunchKernelGGL(head_rest_kernel, dim3(static_cast<unsigned>(tokens)), dim3(kThreads), 0, q, h, piece);
    hipLaunchKernelGGL(head_dx_kernel<BN>, dim3(static_cast<unsigned>(up_to(s.dx_groups, 8))), dx_threads, 0, q, h, piece);
    hipLaunchKernelGGL(head_dx_sum_kernel<BN>, dim3(static_cast<unsigned>(dx_m * n_tiles * DxTile<BN>::NI * DxTile<BN>::NJ * 4)),
                       dx_threads, 0, q, h, piece, static_cast<uint16_t*>(a.dx));
    // dW: into the packed buffer, or with more than one piece into fp32 sums that the last piece rounds
    const dim3 dw(static_cast<unsigned>(std::min<int64_t>(up_to(dx_m * (s.vp / DwTile::kN), 8), kCus)));
    const int64_t start = a.tensor;
    float* sums = reinterpret_cast<float*>(static_cast<char*>(a.work) + s.acc);
    const float* in = i ? (s.sums ? sums : static_cast<const float*>(a.packed) + start) : a.prev ? a.prev + start : nullptr;
    const dim3 wide(DwTile::kThreads);
    if (two)
      hipLaunchKernelGGL((head_dw_kernel<true, false>), dw, wide, 0, q, h, piece, sigma, in, static_cast<void*>(static_cast<float*>(a.packed) + start));
    else if (s.sums && i + 1 < s.n_pieces)
      hipLaunchKernelGGL((head_dw_kernel<false, false>), dw, wide, 0, q, h, piece, sigma, in, static_cast<void*>(sums));
    else
      hipLaunchKernelGGL((head_dw_kernel<false, true>), dw, wide, 0, q, h, piece, sigma, in,
                         static_cast<void*>(static_cast<uint16_t*>(a.packed) + start));
  }
}

// No tokens: the gradient of the table is zero. Four elements a thread.
template <bool OUT16>
__global__ __launch_bounds__(kThreads) void head_none_kernel(const float* prev, void* packed, int64_t n) {
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4;
  for (int64_t i = first; i < n && i < first + 4; ++i) {
    const float y = prev ? prev[i] + 0.0f : 0.0f;
    if constexpr (OUT16) static_cast<uint16_t*>(packed)[i] = static_cast<uint16_t>(bf16_rne(y));
    else static_cast<float*>(packed)[i] = y;
  }
}

int run_head(rs_plan* p, HeadArgs a, bool grad, void* stream, const char* who) {
  clear_error();
  int st = check_call(p, who);
  HeadShape s;
  if (st == RS_OK) st = head_shape(p, a.tensor, a.n, a.top, grad, grad ? a.packed_dt : RS_F32, a.piece, who, &s);
  if (st != RS_OK) return st;
  if (!a.gathered || (a.n && (!a.x || !a.ids || !a.loss || !a.work)) || (grad && (!a.packed || (a.n && !a.dx))))
    return fail(RS_EINVAL, std::string(who) + ": null argument");
  if (a.id_bytes != 4 && a.id_bytes != 8) return fail(RS_EINVAL, std::string(who) + ": token ids have 4 or 8 bytes");
  if (reinterpret_cast<uintptr_t>(a.ids) % static_cast<uintptr_t>(a.id_bytes))
    return fail(RS_EALIGN, std::string(who) + ": token ids must be aligned to their size");
  if ((a.teacher_dt != RS_F32 && a.teacher_dt != RS_BF16) || (grad && a.packed_dt != RS_F32 && a.packed_dt != RS_BF16))
    return fail(RS_EDTYPE, std::string(who) + ": fp32 or bf16");
  if (!std::isfinite(a.scale) || !(a.temperature > 0.0f) || !std::isfinite(a.temperature) || !std::isfinite(a.scale / a.temperature) ||
      !std::isfinite(a.temperature * a.temperature) || !(a.temperature * a.temperature > 0.0f))
    return fail(RS_EINVAL, std::string(who) + ": scale and scale / temperature must be finite, temperature and its square finite and above 0");
  if (grad && !std::isfinite(a.temperature * a.scale))
    return fail(RS_EINVAL, std::string(who) + ": temperature * scale must be finite");
  if (grad && a.prev == a.packed && a.packed_dt != RS_F32)
    return fail(RS_EINVAL, std::string(who) + ": prev may be packed only when packed is fp32");
  if (grad && ((a.scale_mode != RS_SCALE_INV_V && a.scale_mode != RS_SCALE_GIVEN) || !std::isfinite(a.grad_scale)))
    return fail(RS_EINVAL, std::string(who) + ": bad scale");
  for (const void* b : {a.gathered, a.x, static_cast<const void*>(a.loss), static_cast<const void*>(a.weights), static_cast<const void*>(a.dx),
                        static_cast<const void*>(a.prev), static_cast<const void*>(a.packed), static_cast<const void*>(a.work), a.teacher})
    if (!aligned16(b)) return fail(RS_EALIGN, std::string(who) + ": buffers must be 16-byte aligned");
  if (a.work_bytes < s.bytes)
    return fail(RS_EINVAL, std::string(who) + ": workspace of " + std::to_string(a.work_bytes) + " bytes, " + std::to_string(s.bytes) +
                               " needed");
  hipStream_t q = static_cast<hipStream_t>(stream);
  const Tensor& t = p->t[a.tensor];
  const float sigma = a.scale_mode == RS_SCALE_INV_V ? static_cast<float>(static_cast<double>(a.grad_scale) / static_cast<double>(p->V))
                                                     : a.grad_scale;
  if (a.n == 0) {
    if (!grad || a.prev == a.packed) return RS_OK;
    const dim3 grid(static_cast<unsigned>((t.n + kThreads * 4 - 1) / (kThreads * 4)));
    const float* prev = a.prev ? a.prev + t.start : nullptr;
    if (a.packed_dt == RS_BF16)
      hipLaunchKernelGGL(head_none_kernel<true>, grid, dim3(kThreads), 0, q, prev, static_cast<void*>(static_cast<uint16_t*>(a.packed) + t.start), t.n);
    else
      hipLaunchKernelGGL(head_none_kernel<false>, grid, dim3(kThreads), 0, q, prev, static_cast<void*>(static_cast<float*>(a.packed) + t.start), t.n);
    return launched(who);
  }
  char* w = static_cast<char*>(a.work);
  const char* table = static_cast<const char*>(a.gathered) + t.start * 2;
  Head h{};
  h.n = static_cast<int32_t>(s.n);
  h.npad = static_cast<int32_t>(s.npad);
  h.rows = static_cast<int32_t>(s.rows);
  h.cols = static_cast<int32_t>(s.cols);
  h.vp = static_cast<int32_t>(s.vp);
  h.hp = static_cast<int32_t>(s.hp);
  h.top = static_cast<int32_t>(s.top);
  h.piece = static_cast<int32_t>(s.piece);
  h.table = s.widen ? w + s.table : table;
  h.pitch = static_cast<int32_t>(s.hp * 2);
  h.table_bytes = s.rows * s.hp * 2;
  h.info = reinterpret_cast<HeadInfo*>(w + s.info);
  h.pieces = reinterpret_cast<HeadPiece*>(w + s.pieces);
  h.keep = reinterpret_cast<uint32_t*>(w + s.keep);
  h.xmax = reinterpret_cast<float*>(w + s.xmax);
  h.ent = reinterpret_cast<float*>(w + s.ent);
  h.idx = reinterpret_cast<int32_t*>(w + s.idx);
  h.q = reinterpret_cast<float*>(w + s.q);
  h.kept = reinterpret_cast<int32_t*>(w + s.kept);
  h.pent = reinterpret_cast<float*>(w + s.pent);
  h.a = reinterpret_cast<float*>(w + s.a);
  h.lse = reinterpret_cast<float2*>(w + s.lse);
  h.pidx = reinterpret_cast<int32_t*>(w + s.pidx);
  h.pq = reinterpret_cast<float*>(w + s.pq);
  h.picked = reinterpret_cast<float*>(w + s.picked);
  h.xb = w + s.xb;
  h.xh = w + s.xh;
  h.stat = reinterpret_cast<float2*>(w + s.stat);
  h.logits = reinterpret_cast<float*>(w + s.logits);
  h.d = reinterpret_cast<uint16_t*>(w + s.d);
  h.slabs = w + s.slabs;
  h.rest = reinterpret_cast<float*>(w + s.rest);
  h.fix = reinterpret_cast<float*>(w + s.fix);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  const float factor = a.temperature * a.scale;   // f c
  const dim3 targets(static_cast<unsigned>((s.n + kThreads / kWave - 1) / (kThreads / kWave)));
  if (grad)
    hipLaunchKernelGGL(head_targets_kernel<true>, targets, dim3(kThreads), 0, q, h, a.ids, a.id_bytes == 8, a.teacher, a.teacher_dt == RS_BF16,
                       a.temperature, x, a.loss, static_cast<uint16_t*>(a.dx));
  else
    hipLaunchKernelGGL(head_targets_kernel<false>, targets, dim3(kThreads), 0, q, h, a.ids, a.id_bytes == 8, a.teacher, a.teacher_dt == RS_BF16,
                       a.temperature, x, a.loss, static_cast<uint16_t*>(nullptr));
  hipLaunchKernelGGL(head_keep_kernel, dim3(1), dim3(kKeepThreads), 0, q, h, a.weights, factor, static_cast<int>(s.n_pieces),
                     static_cast<int>((s.cols + kTileM - 1) / kTileM), s.tile_n);
  if (grad)
    hipLaunchKernelGGL(head_gather_kernel<true>, dim3(static_cast<unsigned>(s.npad)), dim3(kThreads), 0, q, h, x, a.weights, factor);
  else
    hipLaunchKernelGGL(head_gather_kernel<false>, dim3(static_cast<unsigned>(s.npad)), dim3(kThreads), 0, q, h, x, a.weights, factor);
  if (s.widen)
    hipLaunchKernelGGL(head_widen_kernel, dim3(static_cast<unsigned>((s.rows * (s.hp / 8) + kThreads - 1) / kThreads)), dim3(kThreads), 0, q,
                       reinterpret_cast<const uint16_t*>(table), static_cast<int>(s.rows), static_cast<int>(s.cols), static_cast<int>(s.hp),
                       reinterpret_cast<uint16_t*>(w + s.table));
  a.tensor = t.start;   // elements from here on
  if (s.tile_n == 64) launch_head<64>(s, h, a, sigma, grad, factor, q);
  else if (s.tile_n == 128) launch_head<128>(s, h, a, sigma, grad, factor, q);
  else launch_head<256>(s, h, a, sigma, grad, factor, q);
  return launched(who);
}

}  // namespace
}  // namespace rs

using namespace rs;

extern "C" int rs_head_workspace(const rs_plan* p, int64_t tensor, int64_t n_tokens, int64_t top, int32_t grad, int32_t packed_dt,
                                 int64_t piece, int64_t* bytes) {
  const char* who = "rs_head_workspace";
  clear_error();
  if (!p || !bytes) return fail(RS_EINVAL, std::string(who) + ": null argument");
  if (grad != 0 && grad != 1) return fail(RS_EINVAL, std::string(who) + ": grad is 0 or 1");
  if (packed_dt != RS_F32 && packed_dt != RS_BF16) return fail(RS_EDTYPE, std::string(who) + ": fp32 or bf16");
  HeadShape s;
  const int st = head_shape(p, tensor, n_tokens, top, grad == 1, packed_dt, piece, who, &s);
  if (st != RS_OK) return st;
  *bytes = s.bytes;
  return RS_OK;
}

extern "C" int rs_head_loss(rs_plan* p, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens, const void* targets,
                            int32_t id_bytes, float scale, float* loss, int64_t piece, void* work, int64_t work_bytes, void* stream) {
  const HeadArgs a = {tensor, gathered, x, n_tokens, targets, id_bytes, nullptr, RS_F32, 0, 1.0f, scale, loss, nullptr, nullptr, nullptr,
                      nullptr, RS_F32, RS_SCALE_GIVEN, 1.0f, piece, work, work_bytes};
  return run_head(p, a, false, stream, "rs_head_loss");
}

extern "C" int rs_head_grad(rs_plan* p, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens, const void* targets,
                            int32_t id_bytes, const float* weights, float scale, float* loss, void* dx, const float* prev, void* packed,
                            int32_t packed_dt, int32_t scale_mode, float grad_scale, int64_t piece, void* work, int64_t work_bytes,
                            void* stream) {
  const HeadArgs a = {tensor, gathered, x, n_tokens, targets, id_bytes, nullptr, RS_F32, 0, 1.0f, scale, loss, weights, dx, prev,
                      packed, packed_dt, scale_mode, grad_scale, piece, work, work_bytes};
  return run_head(p, a, true, stream, "rs_head_grad");
}

extern "C" int rs_distill_loss(rs_plan* p, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens, const void* ids,
                               int32_t id_bytes, const void* teacher, int32_t teacher_dt, int64_t top, float temperature, float scale,
                               float* loss, int64_t piece, void* work, int64_t work_bytes, void* stream) {
  const char* who = "rs_distill_loss";
  clear_error();
  if (top < 1 || (n_tokens && !teacher)) return fail(RS_EINVAL, std::string(who) + ": 1 to 256 top logits of a teacher");
  const HeadArgs a = {tensor, gathered, x, n_tokens, ids, id_bytes, teacher, teacher_dt, top, temperature, scale, loss, nullptr, nullptr,
                      nullptr, nullptr, RS_F32, RS_SCALE_GIVEN, 1.0f, piece, work, work_bytes};
  return run_head(p, a, false, stream, who);
}

extern "C" int rs_distill_grad(rs_plan* p, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens, const void* ids,
                               int32_t id_bytes, const void* teacher, int32_t teacher_dt, int64_t top, const float* weights,
                               float temperature, float scale, float* loss, void* dx, const float* prev, void* packed, int32_t packed_dt,
                               int32_t scale_mode, float grad_scale, int64_t piece, void* work, int64_t work_bytes, void* stream) {
  const char* who = "rs_distill_grad";
  clear_error();
  if (top < 1 || (n_tokens && !teacher)) return fail(RS_EINVAL, std::string(who) + ": 1 to 256 top logits of a teacher");
  const HeadArgs a = {tensor, gathered, x, n_tokens, ids, id_bytes, teacher, teacher_dt, top, temperature, scale, loss, weights, dx, prev,
                      packed, packed_dt, scale_mode, grad_scale, piece, work, work_bytes};
  return run_head(p, a, true, stream, who);
}
