/*
 * rs.h — RaggedShard / DBuffer layout transforms on one MI355X (gfx950).
 *
 * A group of N tensors shares one flat buffer of V*S elements; logical rank k
 * owns the slice [k*S, (k+1)*S). Tensor i occupies the contiguous interval
 * [s_i, s_i + n_i); intervals are disjoint and padding lives only between
 * them; a rank boundary that falls inside a tensor falls between two of its
 * atomic blocks ("veScale-FSDP: flexible, structure-aware sharding at
 * 10K-GPU scale", feynmanwiki walkthrough: the paragraphs on RaggedShard's
 * forbidden cut and on the planner as a packing problem). The V ranks are
 * slices of one GPU buffer: nothing here runs a collective.
 *
 * Calls (all extern "C", all return rs_status unless noted):
 *   rs_plan_build       host planner: S and the starts s_i
 *   rs_plan_load        validate a plan and lower it to device work lists
 *   rs_plan_load_with   the same, with options
 *   rs_plan_info / rs_plan_free
 *   rs_unpack_gathered  gathered flat buffer -> N full tensors
 *   rs_pack_scatter     N full gradients -> flat buffer, fused scale/add/zero
 *   rs_block_quant      per-block absmax 8-bit quantisation of the flat buffer
 *   rs_block_quant_noalloc  the same from the plan as data, with its work list
 *                       in static device memory (no allocation)
 *   rs_block_dequant    the inverse of rs_block_quant
 *   rs_unpack_dequant   gathered codes + scales -> the quantised full tensors
 *   rs_adam8_step       one AdamW step on block-quantised int8 / uint8 state
 *   rs_embed_rows       embedding lookup straight from the gathered buffer
 *   rs_embed_grad       its gradient straight into the packed buffer
 *   rs_embed_workspace  bytes of workspace rs_embed_grad needs
 *   rs_layer_norm       layer norm (or RMS norm) with its weight and bias in
 *                       the gathered buffer
 *   rs_layer_norm_grad  its gradient, the parameters' straight into the
 *                       packed buffer
 *   rs_layer_norm_workspace  bytes of workspace rs_layer_norm_grad needs
 *   rs_head_loss        softmax cross entropy of a vocabulary head whose table
 *                       is in the gathered buffer, without handing out logits
 *   rs_head_grad        the same with its gradients, the table's straight into
 *                       the packed buffer
 *   rs_distill_loss     divergence of that head from a teacher's top logits
 *   rs_distill_grad     the same with its gradients
 *   rs_head_workspace   bytes of workspace these four need
 *   rs_orthogonalize    Newton-Schulz orthogonalisation of the WHOLE matrices
 *   rs_muon_step        one Muon step on the WHOLE matrices
 *   rs_muon_workspace   bytes of workspace the two need
 *   rs_last_error       text of the calling thread's last error
 *
 * Conventions
 *   - Sizes and offsets are in elements unless a name says bytes; all int64.
 *   - Device pointers come from the caller (e.g. torch tensors' data_ptr())
 *     and stay owned by the caller. The library owns rs_plan and the device
 *     tables it allocates once in rs_plan_load; no transform call allocates.
 *     rs_block_quant_noalloc allocates nothing at all: its work list goes
 *     into a static device array.
 *   - `stream` is a hipStream_t passed as void* (torch's current stream on
 *     ROCm). Transform calls are asynchronous and ordered on that stream.
 *   - Every check happens before any launch: on error nothing is enqueued,
 *     the status is returned and rs_last_error() says why. No C++ exception
 *     crosses this boundary.
 *   - A plan caches the per-tensor pointer tables it last saw and uploads a
 *     new table on `stream` only when they change; kernels read the table
 *     when they run. The upload is ordered with the work on `stream` only.
 *     A plan is therefore not safe to use from two threads at once; and when
 *     its calls go to more than one stream, a call with new tensor pointers
 *     must be ordered after every earlier call on the other streams, and the
 *     later calls on other streams after it (an event or a synchronisation).
 *   - HIP graphs: the transform calls may be captured (hipStreamBeginCapture
 *     on `stream`) once a call with the same tensor pointers has run outside
 *     the capture and is ordered before the replays. The graph then holds
 *     kernel launches only; they read the plan's pointer table when they run.
 *     A call whose pointers differ from the plan's last call returns
 *     RS_EINVAL while its stream is capturing, and launches nothing. Calls
 *     with other pointers between replays change the tables the replays
 *     read: keep them fixed while such a graph is in use, or use a second
 *     plan for other tensors.
 *   - Floating-point inputs must be finite; NaN or Inf inside a quantisation
 *     block gives unspecified codes (padding is never read, so it may hold
 *     anything).
 */
#ifndef RS_H
#define RS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rs_status {
  RS_OK = 0,
  RS_EINVAL = -1,   /* bad argument: null pointer, n < 1, V < 1, unknown enum ... */
  RS_EPLAN = -2,    /* the plan breaks a constraint, or no plan exists */
  RS_EALIGN = -3,   /* a pointer is not 16-byte aligned, or S / a start not a multiple of 16 */
  RS_EDTYPE = -4,   /* dtype or code format not supported by this call */
  RS_ENOMEM = -5,   /* host or device allocation failed (rs_plan_load only) */
  RS_EHIP = -6,     /* a HIP runtime call or a kernel launch failed */
  RS_ERANGE = -7    /* int64 overflow, or R_mat outside [R_used, V] */
} rs_status;

typedef enum rs_dtype {
  RS_F32 = 0,
  RS_BF16 = 1,
  RS_E4M3 = 2,      /* OCP FP8 E4M3 (largest finite 448, no infinities) */
  RS_I8 = 3,        /* signed, symmetric [-127, 127] */
  RS_U8 = 4         /* unsigned [0, 255] */
} rs_dtype;

/* Atomic block of a tensor: the unit a rank boundary may never cut
 * (feynmanwiki walkthrough, RaggedShard paragraphs: one element, rows, or a
 * larger custom block). The flat block size g follows from the kind:
 *   RS_ELEM        one element                        g = 1
 *   RS_ROWS(k)     k whole rows                       g = k * cols
 *   RS_TILE(br,bc) br x bc tiles of the row-major tensor; a rank boundary may
 *                  only fall between br-row bands (the walkthrough's 8-bit
 *                  Adam: 32x32 blocks at 32-row granularity)   g = br * cols
 *   RS_FLAT(b)     b consecutive elements             g = b
 *   RS_WHOLE       the whole tensor (one matrix per rank, as Muon wants)
 *                                                     g = rows * cols
 *   RS_TILEMAJOR(br,bc) br x bc tiles stored tile by tile: in the flat buffer
 *                  the tensor is its tiles in tile-row-major order, each tile
 *                  contiguous and row-major inside, so a rank boundary may
 *                  fall between any two tiles (the walkthrough's 2-D blocks
 *                  distributed asymmetrically)           g = br * bc
 *                  Needs rows % br == 0, cols % bc == 0, br*bc % 16 == 0 and
 *                  bc <= 8192. Unpack and pack reorder between this layout and
 *                  the row-major tensor (staged through LDS on the GPU).
 * The last block of a tensor may be partial. TILE, TILEMAJOR and FLAT
 * tensors are the ones rs_block_quant quantises (tiles / flat blocks); the
 * others are not. */
typedef enum rs_block_kind {
  RS_ELEM = 0, RS_ROWS = 1, RS_TILE = 2, RS_FLAT = 3, RS_WHOLE = 4, RS_TILEMAJOR = 5
} rs_block_kind;

/* One tensor of the group. A 1-D tensor of n elements is rows = n, cols = 1.
 * p0: ROWS k, TILE br, FLAT b; p1: TILE bc; unused fields must be 0.
 * Limits: rows * cols <= 2^40; a tile (br * bc) or a flat block (b) holds at
 * most 2^24 elements. */
typedef struct rs_tensor_spec {
  int64_t rows;
  int64_t cols;
  int32_t kind;      /* rs_block_kind */
  int32_t reserved;  /* must be 0 */
  int64_t p0;
  int64_t p1;
} rs_tensor_spec;

typedef struct rs_plan rs_plan;   /* opaque, owned by the library */

enum { RS_ORDER_BEST = 0, RS_ORDER_DEFAULT = 1, RS_ORDER_BLOCK_SIZE = 2, RS_ORDER_SHAPE = 3 };
enum { RS_ORDER_KIND_DEFAULT = 0, RS_ORDER_KIND_BLOCK = 1, RS_ORDER_KIND_SHAPE = 2 };

/* Host planner (feynmanwiki walkthrough: the planner paragraphs on the
 * tensor order, on one candidate per-device size and on the search over
 * sizes; bud-325 summary, Method (2)).
 * For each tensor order tried — the caller's order, block size descending,
 * shape descending (element count, then rows), all stable — find the
 * smallest S that is a multiple of `align` and at least
 *   LB = align_up(max(ceil(sum n_i / V), max_i min(g_i, n_i)), align)
 * for which placing each tensor at its earliest valid start after the
 * previous tensor's end fits inside V*S. Keep the order with the smallest S,
 * then the smallest end max(s_i + n_i), then the one listed first.
 * policy: RS_ORDER_BEST tries the three orders; RS_ORDER_DEFAULT,
 * RS_ORDER_BLOCK_SIZE or RS_ORDER_SHAPE plans with that one order (to compare
 * the orders). align >= 1 (16 for plans that rs_plan_load accepts).
 * Outputs (caller-owned host arrays): *S_out; starts_out[n] in the caller's
 * tensor order; order_out[n] the placement order (a permutation of 0..n-1);
 * *order_kind_out one of RS_ORDER_KIND_*. order_out / order_kind_out may be
 * NULL. Host only: touches no GPU.
 * Errors: RS_EINVAL (null, n < 1, V < 1, align < 1, bad spec), RS_ERANGE
 * (int64 overflow). */
int rs_plan_build(const rs_tensor_spec* specs, int64_t n, int64_t V, int64_t align,
                  int32_t policy, int64_t* S_out, int64_t* starts_out,
                  int64_t* order_out, int32_t* order_kind_out);

/* Validate a plan and build its device work lists on `device` (the pages'
 * persistent per-tensor address mapping, made once).
 * R_mat: number of rank slices actually allocated by the caller, with
 * R_used = ceil(max(s_i + n_i) / S) <= R_mat <= V; ranks at or past R_mat
 * hold only padding and are never touched.
 * Checks (RS_EPLAN unless noted): S > 0 and S % 16 == 0 and every
 * s_i % 16 == 0 (RS_EALIGN); intervals disjoint and inside [0, V*S); no
 * rank boundary inside a tensor except at a multiple of g_i from s_i;
 * R_mat in [R_used, V] (RS_ERANGE); V*S fits int64 (RS_ERANGE);
 * R_mat*S <= 2^39 elements and fewer than 2^32 work items per launch
 * (RS_ERANGE; neither limit is reached by a group one device can hold).
 * Environment read here, once per plan: RS_E4M3_ENCODER=sw selects the
 * integer E4M3 encoder instead of gfx950's conversion instruction;
 * RS_TM_KERNEL=direct runs the tile-major reorder of unpack / pack with
 * direct per-lane kernels instead of staging it through LDS. Both give
 * identical results. RS_MUON_TILE=64|128|256 forces the output tile of the
 * matrix products (rs_orthogonalize, rs_muon_step), small matrices included;
 * RS_MUON_PAIRS=1 runs their first two steps together for every matrix whose
 * operands have one part (more than 64 rows and columns); RS_MUON_CUTS=1 cuts
 * every tile of their last, partial round along the contraction.
 * On success *out owns host memory and one device allocation, released by
 * rs_plan_free. Errors: the above, RS_ENOMEM, RS_EHIP. */
int rs_plan_load(const rs_tensor_spec* specs, int64_t n, int64_t V, int64_t S,
                 const int64_t* starts, int64_t R_mat, int32_t device, rs_plan** out);

/* What a plan's calls do that its tensors do not say; all zero is what
 * rs_plan_load takes. */
typedef struct rs_plan_options {
  int32_t muon_parts;   /* fp16 parts of the operands of rs_orthogonalize and rs_muon_step: 1 (or
                         * 0), or 2 for every matrix, for results as near as fp32 products' */
  int32_t reserved[7];  /* must be 0 */
} rs_plan_options;

/* rs_plan_load with options (NULL: none). Errors: as there, and RS_EINVAL for
 * an option outside its values. */
int rs_plan_load_with(const rs_tensor_spec* specs, int64_t n, int64_t V, int64_t S,
                      const int64_t* starts, int64_t R_mat, int32_t device,
                      const rs_plan_options* options, rs_plan** out);

/* Plan facts; any output pointer may be NULL. n_qblocks is the number of
 * quantisation blocks, i.e. the length of rs_block_quant's scale array:
 * tensors in the caller's order; within a TILE tensor its tiles row-major,
 * within a FLAT tensor its blocks in order. padding_elems counts the
 * positions of [0, R_mat*S) that belong to no tensor. */
int rs_plan_info(const rs_plan* plan, int64_t* R_used, int64_t* n_qblocks,
                 int64_t* padding_elems);

void rs_plan_free(rs_plan* plan);   /* NULL is a no-op; waits for the device */

/* Unpack after the (simulated) AllGather: T_i[e] = gathered[s_i + e] for
 * every tensor i and 0 <= e < n_i, bit for bit (for a TILEMAJOR tensor,
 * element (r, c) is read from its place in its tile) (feynmanwiki walkthrough,
 * DBuffer paragraphs: a tensor is its planned slice; this call does the
 * Copy-Out of FSDP2's Copy-Out / Copy-In paragraph in one launch).
 * gathered: device, R_mat*S elements of `dt`, 16-byte aligned.
 * dst: HOST array of n device pointers, each a contiguous row-major tensor of
 * n_i elements of `dt`, 16-byte aligned. dt: RS_F32, RS_BF16 or any 1-byte
 * dtype (RS_E4M3 / RS_I8 / RS_U8). Padding of `gathered` is never read.
 * Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_EHIP. */
int rs_unpack_gathered(rs_plan* plan, const void* gathered, int32_t dt,
                       void* const* dst, void* stream);

enum { RS_SCALE_INV_V = 0, RS_SCALE_GIVEN = 1 };

/* Pack before the (simulated) ReduceScatter, with the group-fused pre-
 * communication ops (feynmanwiki walkthrough, DBuffer paragraph on add,
 * scale, zero and copy fused at group level):
 *   sigma = fl32(1/V) for RS_SCALE_INV_V, else `scale`;
 *   y = fl32(src_i[e] * sigma);
 *   packed[s_i + e] = prev ? fl32(prev[s_i + e] + y) : y
 * (for a TILEMAJOR tensor, element (r, c) goes to its place in its tile)
 * (scale first, then add: two IEEE round-to-nearest-even operations, never a
 * fused multiply-add), and packed[p] = +0.0 at every padding position p in
 * [0, R_mat*S). Padding of `prev` is never read. With packed_dt = RS_BF16
 * (a bf16 ReduceScatter, as in mixed-precision training) each fp32 result
 * is rounded once to the nearest bf16, ties to even.
 * src: HOST array of n device pointers to contiguous gradients (src_dt
 * RS_F32 or RS_BF16, 16-byte aligned). prev: device fp32 R_mat*S or NULL (no
 * accumulation); it may equal `packed` (in-place accumulation) only when
 * packed_dt is RS_F32 (otherwise RS_EINVAL), and must not overlap it in any
 * other way. packed: device R_mat*S elements of packed_dt (RS_F32 or
 * RS_BF16), 16-byte aligned.
 * Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_EHIP. */
int rs_pack_scatter(rs_plan* plan, const void* const* src, int32_t src_dt,
                    const float* prev, void* packed, int32_t packed_dt, int32_t scale_mode,
                    float scale, void* stream);

/* Block-wise quantisation of every locally whole block (feynmanwiki
 * walkthrough, block-quantisation paragraph: all codes of a block depend on
 * one per-block scale, so a rank boundary must never split a block; and the
 * 8-bit Adam paragraph). For each block B
 * (a br x bc tile of a TILE tensor, partial at the edges, or a b-element
 * block of a FLAT tensor):
 *   amax = max |x| over B;  Q = 448 (RS_E4M3), 127 (RS_I8), 255 (RS_U8);
 *   amax == 0: scale[B] = 1.0 and every code is 0;
 *   amax NaN (a NaN in B; NaN wins the max) or +inf (an infinity in B):
 *   scale[B] = quiet NaN 0x7FC00000 or +inf and every code is 0, so the
 *   block dequantises to NaN everywhere (the pages assume finite values);
 *   otherwise scale[B] = fl32(amax / Q), r = min(fl32(Q / amax), FLT_MAX),
 *   code = enc(fl32(x * r)), enc being round-to-nearest-even with saturation
 *   (E4M3: to +-448, sign kept, -0 -> 0x80; I8: to [-127,127]; U8: [0,255]).
 * Every byte of q outside all blocks (padding, untiled tensors) is 0x00.
 * E4M3 codes come from gfx950's FP8 conversion instructions unless the
 * environment variable RS_E4M3_ENCODER=sw is set when the plan is loaded
 * (then an integer encoder is used); both give identical codes.
 * src: device, R_mat*S elements of src_dt (RS_F32 or RS_BF16), 16-byte
 * aligned. q: device, R_mat*S bytes, 16-byte aligned. scales: device fp32
 * [n_qblocks] (rs_plan_info), ordered by tensor, then tile row-major or flat
 * block index.
 * Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_EHIP. */
int rs_block_quant(rs_plan* plan, const void* src, int32_t src_dt, void* q, int32_t q_dt,
                   float* scales, void* stream);

/* Allocation-free variant of rs_block_quant, for callers that cannot
 * allocate device memory (tight serving loops, harnesses that forbid
 * allocation). It takes the plan as data (the arguments of rs_plan_load)
 * instead of a loaded plan: it validates the plan, builds the quant work list
 * on the host and copies it into a static device array of 16 MiB that each GPU
 * holds for the life of the process: at most 262,144 work items, one per
 * tile, per pair of flat blocks and per 65,536 positions outside all blocks.
 * It calls no hipMalloc, hipFree or other allocating HIP routine. Codes and
 * scales equal those of rs_block_quant on the same plan, bit for bit.
 * The work list is copied on `stream`, after the work already queued there,
 * and the call waits for `stream` before it launches. Every call on one GPU
 * shares that GPU's array: calls in order on one stream are safe; calls that
 * may overlap on one GPU (other streams, other host threads) race, and the
 * caller must serialise them.
 * specs, n, V, S, starts, R_mat: as for rs_plan_load; the current device runs
 * the call. src, src_dt, q, q_dt: as for rs_block_quant. scales: device fp32,
 * scales_len entries, at least the plan's number of blocks.
 * Errors: the plan's validation errors as for rs_plan_load, RS_EDTYPE,
 * RS_EALIGN, RS_EINVAL (null buffer, scales too short), RS_ERANGE (work list
 * larger than the static array: load the plan and call rs_block_quant),
 * RS_EHIP. Nothing is launched on an error. */
int rs_block_quant_noalloc(const rs_tensor_spec* specs, int64_t n, int64_t V, int64_t S,
                           const int64_t* starts, int64_t R_mat, const void* src, int32_t src_dt,
                           void* q, int32_t q_dt, float* scales, int64_t scales_len, void* stream);

/* Inverse of rs_block_quant: out[p] = fl32(dec(q[p]) * scale[B]) inside
 * block B, +0.0 everywhere else in [0, R_mat*S). Arguments as in
 * rs_block_quant; out: device fp32 R_mat*S, 16-byte aligned. */
int rs_block_dequant(rs_plan* plan, const void* q, int32_t q_dt, const float* scales,
                     float* out, void* stream);

/* Gather side of block-wise FP8 training, fused (bud-325 summary, TL;DR and
 * Key claims: DeepSeek-V3-style block-wise FP8; feynmanwiki walkthrough,
 * block-quantisation paragraph): after the codes and scales of every rank
 * slice are all-gathered, rebuild each quantised tensor straight from them:
 *   T_i[e] = fl32(dec(q[s_i + e]) * scale[B])   for e in block B of T_i,
 * rounded to bf16 (nearest, ties to even) when dst_dt is RS_BF16. This is
 * rs_block_dequant followed by rs_unpack_gathered (and a cast), in one pass
 * that reads each code once and writes each value once.
 * q, q_dt, scales: as produced by rs_block_quant (device, R_mat*S bytes,
 * 16-byte aligned; fp32 [n_qblocks]). dst: HOST array of n device pointers;
 * entries of TILE, TILEMAJOR and FLAT tensors point to contiguous row-major tensors of
 * n_i elements of dst_dt (RS_BF16 or RS_F32), 16-byte aligned; entries of
 * other tensors are ignored and may be NULL. Codes 0x7F / 0xFF (E4M3 NaN)
 * give unspecified values. Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_EHIP. */
int rs_unpack_dequant(rs_plan* plan, const void* q, int32_t q_dt, const float* scales,
                      void* const* dst, int32_t dst_dt, void* stream);

/* Hyper-parameters of one Adam step; step counts from 1. */
typedef struct rs_adam_hparams {
  float lr;
  float beta1;         /* in [0, 1) */
  float beta2;         /* in [0, 1) */
  float eps;           /* >= 0 */
  float weight_decay;  /* decoupled (AdamW); 0 for plain Adam */
  int32_t reserved;    /* must be 0 */
  int64_t step;        /* >= 1 */
} rs_adam_hparams;

/* One 8-bit Adam step on every quantisation block of the plan, in place
 * (feynmanwiki walkthrough, 8-bit Adam paragraph: optimizer state quantised
 * in blocks that stay whole on their device, so each device updates and
 * requantises its own blocks with no scale exchange). The pages give no
 * update formula; this is AdamW. Host scalars, computed in double from the
 * fp32 hyper-parameters and rounded once to fp32:
 *   c1 = 1 - b1, c2 = 1 - b2, step_size = lr / (1 - b1^t),
 *   inv_bc2_sqrt = 1 / sqrt(1 - b2^t), decay = 1 - lr*wd.
 * Per element of a block B, each operation one fp32 round-to-nearest-even
 * step (no fused multiply-add):
 *   m0 = dec_i8(q_m) * s_m[B]        v0 = dec_u8(q_v) * s_v[B]
 *   m1 = b1*m0 + c1*g                v1 = b2*v0 + c2*(g*g)
 *   den = sqrt(v1)*inv_bc2_sqrt + eps
 *   param = param*decay - step_size*(m1/den)
 * then m1 and v1 are requantised per block exactly as rs_block_quant does
 * (int8 and uint8). Positions outside quantisation blocks are not touched.
 * param: device fp32 R_mat*S (in place); grad: device fp32 R_mat*S (the
 * packed gradient, e.g. from rs_pack_scatter); q_m / q_v: device int8 / uint8
 * codes, R_mat*S bytes, in place; s_m / s_v: device fp32 [n_qblocks], in
 * place. All 16-byte aligned. hp: host pointer.
 * Errors: RS_EINVAL (null, step < 1, beta outside [0,1), eps < 0, non-finite
 * lr / wd), RS_EALIGN, RS_EHIP. */
int rs_adam8_step(rs_plan* plan, float* param, const float* grad, void* q_m, float* s_m,
                  void* q_v, float* s_v, const rs_adam_hparams* hp, void* stream);

/* Embedding lookup straight from the gathered buffer: what rs_unpack_gathered
 * would copy of one tensor, for the rows that a batch of tokens names
 * (feynmanwiki walkthrough, DBuffer paragraphs: a tensor is its planned
 * slice). With T = tensor `tensor` of the plan, rows x cols:
 *   out[t, c] = fl32(T[ids[t], c] * scale)   for 0 <= t < n_ids,
 * rounded once more to bf16 (nearest, ties to even) when out_dt is RS_BF16.
 * An id outside [0, rows) (padding tokens, e.g. -1) names no row: its output
 * row is +0.0. Any block kind but RS_TILEMAJOR (whose rows are not
 * contiguous).
 * gathered: device, R_mat*S elements of dt (RS_F32 or RS_BF16). ids: device,
 * n_ids signed integers of id_bytes (4 or 8) bytes. scale: finite. out:
 * device, n_ids x cols row-major of out_dt (RS_F32 or RS_BF16), overlapping
 * neither input. gathered and out 16-byte aligned. n_ids may be 0.
 * Limits (RS_ERANGE): rows at most 2^27 - 8, cols under 2^31, rows * cols at
 * most 2^34, n_ids under 2^26, n_ids * cols at most 2^33.
 * Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_ERANGE, RS_EHIP. */
int rs_embed_rows(rs_plan* plan, int64_t tensor, const void* gathered, int32_t dt, const void* ids,
                  int32_t id_bytes, int64_t n_ids, float scale, void* out, int32_t out_dt, void* stream);

/* Gradient of the lookup straight into the packed buffer: what
 * rs_pack_scatter would write of one tensor, without the dense gradient.
 *   y[r, c] = fl32(sigma * sum of dy[t, c] over the t with ids[t] = r)
 *   packed[r, c] = prev ? fl32(prev[r, c] + y[r, c]) : y[r, c]
 * on the tensor's interval of the flat buffers (r, c there), with sigma =
 * scale (RS_SCALE_GIVEN) or fl32(scale / V) (RS_SCALE_INV_V); a bf16 packed
 * buffer gets the result rounded once to nearest even. Sums are fp32, in an
 * order that depends on the ids alone: the same call gives the same bits.
 * Ids outside [0, rows) contribute nothing and their dy is not read.
 * prev = packed (fp32 only) adds in place: rows that no token names are
 * neither read nor written, e.g. a tied table whose dense gradient is packed
 * already. Otherwise every row of the tensor is written (+0.0, or prev + 0.0,
 * where no token names it), and prev must not overlap packed. Positions
 * outside the tensor's interval are left alone in any case.
 * dy: device, n_ids x cols row-major of dy_dt (RS_F32 or RS_BF16). prev:
 * device fp32 R_mat*S or NULL. packed: device R_mat*S of packed_dt (RS_F32 or
 * RS_BF16). work: device memory of rs_embed_workspace bytes, contents not
 * kept between calls; calls that may overlap need a workspace each. All
 * 16-byte aligned; ids and limits as in rs_embed_rows.
 * Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_ERANGE, RS_EHIP. */
int rs_embed_grad(rs_plan* plan, int64_t tensor, const void* ids, int32_t id_bytes, int64_t n_ids,
                  const void* dy, int32_t dy_dt, const float* prev, void* packed, int32_t packed_dt,
                  int32_t scale_mode, float scale, void* work, int64_t work_bytes, void* stream);

/* Bytes of workspace for rs_embed_grad on this tensor with n_ids tokens; it
 * grows with n_ids. Errors: RS_EINVAL, RS_ERANGE. */
int rs_embed_workspace(const rs_plan* plan, int64_t tensor, int64_t n_ids, int64_t* bytes);

/* Layer norm of each row of x with its parameters where the gather left them
 * (feynmanwiki walkthrough, DBuffer paragraphs: a tensor is its planned
 * slice). With C the number of elements of tensor `weight`, w its elements and
 * b those of tensor `bias` (0 where bias is -1), per row:
 *   m = center ? sum(x) / C : 0
 *   r = 1 / sqrt(sum((x - m)^2) / C + eps)
 *   y = (x - m) r w + b
 * center 0 is the RMS norm. Sums and all steps are fp32, in an order that
 * depends on C alone; a bf16 y is rounded once, to nearest even. A row of zeros
 * gives b (NaN with eps = 0); a NaN or an infinity in a row, or a sum past
 * fp32's range, stays in its row.
 * weight, bias: numbers of two tensors of the plan with the same number of
 * elements, any kind but RS_TILEMAJOR. gathered: device, R_mat*S elements of
 * dt. x: device, n_rows x C row-major of x_dt. y: device, n_rows x C of y_dt,
 * overlapping neither input. All RS_F32 or RS_BF16, 16-byte aligned. n_rows may
 * be 0. eps: finite, >= 0. Limits (RS_ERANGE): C at most 16384, n_rows under
 * 2^31. Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_ERANGE, RS_EHIP. */
int rs_layer_norm(rs_plan* plan, int64_t weight, int64_t bias, const void* gathered, int32_t dt, const void* x,
                  int32_t x_dt, int64_t n_rows, float eps, int32_t center, void* y, int32_t y_dt, void* stream);

/* Gradients of rs_layer_norm from that of y; nothing is kept from the forward
 * call. With h = (x - m) r and g = dy w, per row:
 *   dx = r (g - (center ? sum(g) / C : 0) - h sum(g h) / C)
 * and on the intervals of the two tensors in the packed buffer
 *   weight:  packed = [prev +] sigma * sum over the rows of dy h
 *   bias:    packed = [prev +] sigma * sum over the rows of dy
 * with sigma = scale (RS_SCALE_GIVEN) or fl32(scale / V) (RS_SCALE_INV_V). The
 * sums are fp32, in an order that depends on n_rows and C alone. Both intervals
 * are written whole (also for n_rows = 0); other positions are left alone.
 * x, x_dt, dy (n_rows x C of dy_dt): inputs. dx: device, n_rows x C of x_dt.
 * prev: device fp32 R_mat*S or NULL; it may equal packed (fp32 only) to add in
 * place, and must not overlap it in any other way. packed: device R_mat*S of
 * packed_dt (RS_F32 or RS_BF16). work: device memory of
 * rs_layer_norm_workspace bytes, contents not kept between calls; calls that
 * may overlap need a workspace each. All 16-byte aligned; outputs overlap
 * neither inputs nor each other. Limits and errors as in rs_layer_norm. */
int rs_layer_norm_grad(rs_plan* plan, int64_t weight, int64_t bias, const void* gathered, int32_t dt, const void* x,
                       int32_t x_dt, const void* dy, int32_t dy_dt, int64_t n_rows, float eps, int32_t center, void* dx,
                       const float* prev, void* packed, int32_t packed_dt, int32_t scale_mode, float scale, void* work,
                       int64_t work_bytes, void* stream);

/* Bytes of workspace for rs_layer_norm_grad on n_rows rows, or fewer. Errors:
 * RS_EINVAL, RS_ERANGE. */
int rs_layer_norm_workspace(const rs_plan* plan, int64_t weight, int64_t n_rows, int64_t* bytes);

/* Softmax cross entropy of a vocabulary head, straight from the gathered
 * buffer (feynmanwiki walkthrough, DBuffer paragraphs: a tensor is its planned
 * slice). With W = tensor `tensor` of the plan, rows x cols, and y = targets[t]:
 *   l = scale * (W x_t),   loss[t] = log(sum over r of exp(l_r)) - l_y
 * A target outside [0, rows) (e.g. -100) is none: its loss is +0.0, its x is
 * not read, and it costs next to nothing. The logits live in the workspace at
 * most. Products of bf16 values with fp32 sums; everything else is fp32, with the
 * largest logit taken out first, so a loss is never negative. Sums have a fixed
 * order: the same call gives the same bits. A NaN or an infinity
 * in x_t makes loss[t] NaN (one in W may make all of them NaN).
 * Any block kind but RS_TILEMAJOR. gathered: device, R_mat*S bf16 elements. x:
 * device, n_tokens x cols bf16, row-major. targets: device, n_tokens signed
 * integers of id_bytes (4 or 8) bytes, aligned to their size. scale: finite.
 * loss: device, n_tokens fp32. piece: tokens worked on at a time, a multiple of
 * 256 up to 65536, or 0 for up to 8192; it bounds the workspace, and results
 * may differ in the last bits with it. work: device memory of rs_head_workspace
 * bytes, contents not kept between calls; calls that may overlap need a
 * workspace each. All but targets 16-byte aligned; outputs and workspace
 * overlap neither inputs nor each other. n_tokens may be 0.
 * Limits (RS_ERANGE): n_tokens at most 2^20, rows 2^21, cols 2^16, rows * cols
 * and n_tokens * cols 2^33, n_tokens * top 2^28.
 * Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_ERANGE, RS_EHIP. */
int rs_head_loss(rs_plan* plan, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens,
                 const void* targets, int32_t id_bytes, float scale, float* loss, int64_t piece, void* work,
                 int64_t work_bytes, void* stream);

/* The losses of rs_head_loss and the gradients of sum over t of w_t * loss[t],
 * w_t = weights[t] (1 where weights is NULL). With p the softmax of l, e_y the
 * unit vector of the target and a_t = w_t * scale:
 *   dx_t = a_t * W^T (p - e_y), rounded once to bf16
 *   packed = [prev +] sigma * sum over t of a_t * (p - e_y) x_t^T
 * on W's interval, sigma = grad_scale (RS_SCALE_GIVEN) or fl32(grad_scale / V)
 * (RS_SCALE_INV_V). A token without a target gets a dx of +0.0 and adds nothing,
 * and neither does one of weight 0, whatever its x holds. p - e_y is computed in
 * fp32; for dx it is rounded to bf16 (8 bits), and what that leaves at the target is
 * added in fp32. For the table's gradient a_t (p - e_y) is rounded to 11 bits (a
 * bf16 packed buffer) or 22 (fp32), or to within 2^-38 of the largest |a_t| where
 * that is more, and x to within 2^-38 of the largest |x| of a token of weight not 0
 * (its bf16 values are exact down to 2^-28 of it). Sums are fp32.
 * W's interval is written whole (with n_tokens = 0 too; with prev = packed and
 * no targets it is left alone); other positions are left alone.
 * weights: device, n_tokens fp32, or NULL. dx: device, n_tokens x cols bf16.
 * prev: device fp32 R_mat*S or NULL; it may equal packed (fp32 only) to add in
 * place, and must not overlap it in any other way. packed: device R_mat*S of
 * packed_dt (RS_F32 or RS_BF16). The rest, limits and errors as above. */
int rs_head_grad(rs_plan* plan, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens,
                 const void* targets, int32_t id_bytes, const float* weights, float scale, float* loss, void* dx,
                 const float* prev, void* packed, int32_t packed_dt, int32_t scale_mode, float grad_scale, int64_t piece,
                 void* work, int64_t work_bytes, void* stream);

/* Distillation of the same head from the `top` (1 to 256) largest logits that
 * a teacher gave each token: teacher[t, k] for row ids[t, k] of the table. With
 * T = temperature, l as above and q the softmax of teacher[t] / T over the
 * token's places:
 *   loss[t] = T^2 * sum over k of q_k * (log q_k - log softmax(l / T)[ids[t, k]])
 * Places whose id is outside [0, rows) or whose logit is -inf are empty; a token
 * with none left is one without a target, as above. A row named twice counts
 * with both its shares. A teacher's logit of NaN or +inf makes the token's loss
 * NaN. ids: device, n_tokens x top integers of id_bytes; teacher: device,
 * n_tokens x top of teacher_dt (RS_F32 or RS_BF16), 16-byte aligned.
 * temperature: finite, above 0, as is its square; scale / temperature finite.
 * The rest as in rs_head_loss. */
int rs_distill_loss(rs_plan* plan, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens, const void* ids,
                    int32_t id_bytes, const void* teacher, int32_t teacher_dt, int64_t top, float temperature, float scale,
                    float* loss, int64_t piece, void* work, int64_t work_bytes, void* stream);

/* The losses of rs_distill_loss and the gradients of their weighted sum as in
 * rs_head_grad, with p = softmax(l / T), q in e_y's place and
 * a_t = w_t * T * scale, of which T * scale has to be finite. The teacher's logits
 * get no gradient. */
int rs_distill_grad(rs_plan* plan, int64_t tensor, const void* gathered, const void* x, int64_t n_tokens, const void* ids,
                    int32_t id_bytes, const void* teacher, int32_t teacher_dt, int64_t top, const float* weights,
                    float temperature, float scale, float* loss, void* dx, const float* prev, void* packed,
                    int32_t packed_dt, int32_t scale_mode, float grad_scale, int64_t piece, void* work, int64_t work_bytes,
                    void* stream);

/* Bytes of workspace for the four calls on this tensor with n_tokens tokens, or
 * fewer: piece and top (0 for labels) as in the call; grad 1 for the gradients (a workspace that
 * also serves the losses), packed_dt the packed buffer's type. About
 * 4 n cols + 16 n top for the tokens; rows * cols * 2 more where cols is no
 * multiple of 64; piece * rows * 4 where rows < 256 top, piece * rows * 6 for
 * gradients; for these too piece * cols * 4, as much again or at most 256 MiB for
 * parts of dx,
 * and rows * cols * 4 for a bf16 packed buffer and more than one piece.
 * Errors: RS_EINVAL, RS_EDTYPE, RS_ERANGE. */
int rs_head_workspace(const rs_plan* plan, int64_t tensor, int64_t n_tokens, int64_t top, int32_t grad, int32_t packed_dt,
                      int64_t piece, int64_t* bytes);

/* Orthogonalisation of every matrix of the plan by Newton-Schulz products
 * (feynmanwiki walkthrough, Muon paragraphs: the rank that holds a matrix
 * whole runs Newton-Schulz on it, which is what RS_WHOLE blocks are for). A
 * matrix is a WHOLE tensor of more than one row and one column; other tensors
 * and padding are neither read nor written. For each matrix G (X is G, or its
 * transpose where rows > cols):
 *   X = G / (|G|_F + eps);
 *   for t in 0 .. steps-1:  A = X X^T,  X = (a_t I + b_t A + c_t A^2) X,
 * and out gets X (transposed back) rounded once to the nearest bf16.
 * Products take fp16 operands with fp32 sums; X is carried as a high and a
 * low fp16 part and the diagonals of A and of the polynomial in fp32, which
 * keeps the result within about 1e-3 of the exact one (Frobenius norm), ahead
 * of the bf16 rounding, for polynomials of slopes up to about 2 between 0.3
 * and 1.2, such as the published quintic; steeper ones raise each step's
 * rounding by their slope. Matrices of at most 64 rows or columns, and every
 * matrix of a plan loaded with muon_parts = 2, have all operands in two parts,
 * which keeps the result as near as fp32 products do (5e-7; 1.5e-5 where
 * directions are 100 times weaker than others) at 1.4 to 2.9 times the time.
 * With one part, where that costs less, the first two polynomials
 * (|a| <= 4) are multiplied with each other and applied to X once. The
 * polynomials must keep every singular value below
 * 7 (A is held to 2^16 / 2^10) and the off-diagonal entries of b A + c A^2
 * below 60. The norm is summed in fp64. The sums have a fixed order: the same
 * call gives the same bits. A zero matrix gives zeros; a NaN or an infinity
 * makes its own matrix's result NaN and leaves the others alone.
 * src: device, R_mat*S elements of src_dt (RS_F32 or RS_BF16). out: device
 * bf16, R_mat*S elements, not overlapping src. coeffs: HOST array of 3*steps
 * floats a_t, b_t, c_t (finite). steps: 1 to 32. eps >= 0 (with eps = 0 a
 * zero matrix gives NaN). work: device memory of rs_muon_workspace bytes,
 * whose contents need not be kept between calls; calls that may overlap (on
 * other streams, or in graphs that may) need a workspace each. All 16-byte
 * aligned. Limits (RS_ERANGE): a matrix's sides at most 2^20, one of them at
 * most 2^16, and the matrices of a plan at most 2^22 tiles of 64 x 64.
 * Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_ERANGE, RS_EHIP. */
int rs_orthogonalize(rs_plan* plan, const void* src, int32_t src_dt, void* out, const float* coeffs,
                     int32_t steps, float eps, void* work, int64_t work_bytes, void* stream);

/* Factor on an update's rate: 1; sqrt(max(1, rows/cols)); or
 * 0.2 * sqrt(max(rows, cols)), which gives an orthogonal matrix the root mean
 * square of a usual AdamW update. */
enum { RS_MUON_SCALE_NONE = 0, RS_MUON_SCALE_SPECTRAL = 1, RS_MUON_SCALE_RMS = 2 };

typedef struct rs_muon_hparams {
  float lr;
  float momentum;      /* mu, in [0, 1) */
  float weight_decay;  /* decoupled */
  float eps;           /* >= 0, added to the norm */
  int32_t steps;       /* Newton-Schulz steps, 1 to 32 */
  int32_t nesterov;    /* 0 or 1 */
  int32_t scale_mode;  /* RS_MUON_SCALE_* */
} rs_muon_hparams;

/* One Muon step on every matrix of the plan (see rs_orthogonalize), in place;
 * per matrix, f its factor from scale_mode, all in fp32:
 *   momentum = mu * momentum + grad
 *   U = nesterov ? grad + mu * momentum : momentum
 *   param = param * (1 - lr * weight_decay) - lr * f * orthogonalise(U)
 * The other tensors of the group and the padding are left as they are (they
 * take another optimiser, e.g. rs_adam8_step on their quantisation blocks).
 * A NaN or an infinity in U makes that matrix's parameters NaN.
 * param, momentum: device fp32 R_mat*S, in place. grad: device R_mat*S of
 * grad_dt (RS_F32 or RS_BF16), e.g. from rs_pack_scatter. The three do not
 * overlap. coeffs: HOST array of 3*hp->steps floats. work, work_bytes: as in
 * rs_orthogonalize. Errors: RS_EINVAL, RS_EALIGN, RS_EDTYPE, RS_ERANGE,
 * RS_EHIP. */
int rs_muon_step(rs_plan* plan, float* param, const void* grad, int32_t grad_dt, float* momentum,
                 const rs_muon_hparams* hp, const float* coeffs, void* work, int64_t work_bytes, void* stream);

/* Bytes of workspace that rs_orthogonalize and rs_muon_step need for this
 * plan. All its matrices advance together, so it is a sum over them (a group
 * split over several plans needs the largest of theirs). With m and n a
 * matrix's shorter and longer side, each padded to a multiple of 64, at most:
 *   one part                     8 m n + 4 m^2
 *   one part, m >= 1024 and n >= 1.5 m (the first two steps together)
 *                                8 m n + 8 m^2
 *   two parts                    12 m n + 8 m^2
 *   m <= 64 and n <= 256         nothing
 * and up to 1% and 8 KiB a matrix more for norms, diagonals and alignment, and
 * at most 128 MiB in all for the parts of cut tiles (192 with RS_MUON_CUTS=1).
 * Errors: RS_EINVAL. */
int rs_muon_workspace(const rs_plan* plan, int64_t* bytes);

/* Message for the calling thread's last failed call ("" if none). The
 * pointer stays valid until the thread's next rs_* call. */
const char* rs_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* RS_H */
