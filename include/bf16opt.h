/*
 * bf16opt.h -- C ABI of the MI355X (gfx950) mixed-precision AdamW step.
 *
 * The step has three parts and runs over one ZeRO-1 shard of a flat buffer
 * that holds many tensors back to back:
 *   1. grad_global_norm: a deterministic L2 norm of the bf16 gradients and
 *      the clip scale derived from it;
 *   2. adamw_sr_step: one fused pass per element -- AdamW with lerp-form
 *      moments, bias correction, decoupled weight decay on flagged (2-D)
 *      tensors only, an fp32 master update and a bf16 write-back by
 *      stochastic rounding keyed on (global element index, seed);
 *   3. master_to_bf16_sr: the resume-time rebuild of the bf16 weights from
 *      the fp32 master with the same rounding draws.
 *
 * Pages defining each operation (title, section):
 *   "04 · 多 GPU 与混合精度" (llm.c multi-GPU and mixed precision):
 *     §2.1 precision roles, §2.2 AdamW kernel, §2.3 stochastic rounding,
 *     §3.2 ZeRO-1 sharding, §4 grad norm and clip, §5.2 bit-perfect resume.
 *   "第 13 讲：扩大 LLM——优化与并行训练": §1.7 bias correction and AdamW,
 *     §2.3 fp32 master weights.
 *   "LLM 分布式训练实战：CUDA/ROCm 多卡并行优化详解": §3.1 sharded update.
 *
 * Conventions shared by every entry point
 *   - Shards.  A table describes one rank's shard of the flat buffer, in one
 *     of two layouts.  BFO_LAYOUT_FLAT: the contiguous global range
 *     [begin, end) = [r*n/N, (r+1)*n/N) (see shard_range).  BFO_LAYOUT_PER_TENSOR:
 *     rank r's 1/N slice of every tensor, concatenated in table order (the
 *     llm.c rule that every tensor size divides by the process count).  The
 *     shard holds S elements either way; shard-local element j maps to one
 *     global index i of the flat buffer (bfo_table_runs lists the mapping).
 *   - Arrays.  master, m and v are shard-local: element j of the array
 *     belongs to shard element j; they hold S fp32 values.  params and grads
 *     (bf16 patterns, uint16_t) are addressed differently per layout: FLAT --
 *     shard-local too (element j; pass the full buffer + begin); PER_TENSOR --
 *     the full n-element buffers (element i).
 *   - Memory.  Array arguments are device pointers on the device the table
 *     was created on.  master, m and v must be 16-byte aligned; params and
 *     grads 2-byte aligned (16-byte aligned pointers take the fastest path).
 *     The arrays of one call must not overlap one another (BFO_EINVAL): the
 *     kernels read and write them as distinct buffers.  Scalars and the
 *     hyperparameter struct are host memory.  The caller owns every buffer;
 *     the library keeps no pointer after a call returns.
 *   - Asynchrony.  GPU work is queued on `stream` (a hipStream_t; NULL means
 *     the null stream) and the call returns without waiting for it.  Argument
 *     errors are reported synchronously and queue no work.  Apart from the
 *     checkpoint calls (which move state through files, and so wait for their
 *     copies and use a pinned host stage for the call's length), nothing here
 *     synchronises the host or allocates memory per call; device memory is
 *     allocated only when a table or an outlier detector is created.
 *   - Errors.  Every function returns BFO_OK (0) or a negative BFO_E* code;
 *     bfo_status_string() names it.  BFO_EHIP means a HIP runtime call
 *     failed; bfo_last_hip_error() gives its hipError_t code for the calling
 *     thread.  The library never prints and never exits.
 *   - Concurrency.  A table may be used from several threads and streams;
 *     the one shared buffer is the norm workspace a table holds for callers
 *     that pass none (see grad_global_norm).
 *
 * A step, as a ZeRO-1 rank runs it (error checks left out):
 *   bfo_table tb;  bfo_table_create(tensors, count, world, rank, &tb);   once
 *   bfo_norm_result *res;  (16-byte aligned device memory)              once
 *   void *workspace;  (bfo_norm_workspace_bytes(tb) bytes of device memory) once
 *   per step t = 1, 2, ...:
 *     grad_global_norm(tb, grads + begin, 1.0f, workspace, res, stream);
 *     adamw_sr_step(tb, params + begin, grads + begin, master, m, v, &hp,
 *                   &res->scale, NULL, t, seed_t, BFO_ROUND_SR, stream);
 *   (the all-gather of params and the reduce-scatter of grads around it are
 *   the caller's; every array here is already resident on the device.)
 */
#ifndef BF16OPT_H
#define BF16OPT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    BFO_OK = 0,
    BFO_EINVAL = -1,        /* null pointer, overlapping arrays, world == 0, t == 0, unknown rounding mode */
    BFO_ENOTDIVISIBLE = -2, /* n (or, per tensor, a tensor's size) is not a multiple of world */
    BFO_ERANGE = -3,        /* rank >= world */
    BFO_EMISALIGNED = -4,   /* pointer not aligned as required (see Memory above) */
    BFO_ETABLE = -5,        /* table not contiguous from 0, or undefined flag bits set */
    BFO_EHIP = -6,          /* a HIP runtime call failed */
    BFO_EDEVICE = -7,       /* called with a different current device than the table's */
    BFO_EIO = -8,           /* a checkpoint file could not be created, written or read */
    BFO_EFORMAT = -9,       /* a checkpoint file does not match the table, or is truncated */
    BFO_ENOTFOUND = -10     /* no such checkpoint (file or DONE marker) */
};

enum { BFO_ROUND_SR = 0, BFO_ROUND_RNE = 1 };

enum { BFO_LAYOUT_FLAT = 0, BFO_LAYOUT_PER_TENSOR = 1 };

/* bfo_tensor.flags bit 0: the tensor takes weight decay.  The pages apply
 * decay to 2-D tensors (embeddings, weight matrices) and not to 1-D ones
 * (LayerNorm / RMSNorm weights, biases): "04 · 多 GPU 与混合精度" §2.2. */
#define BFO_FLAG_DECAY 1u

/* One tensor of the flat buffer: global elements [offset, offset + numel).
 * A table lists the tensors in buffer order; tensor k must start where
 * tensor k-1 ends, the first at 0; numel may be 0; `reserved` must be 0. */
typedef struct {
    uint64_t offset;
    uint64_t numel;
    uint32_t flags;
    uint32_t reserved;
} bfo_tensor;

/* AdamW hyperparameters ("04 · 多 GPU 与混合精度" §4: lr, beta1 = 0.9,
 * beta2 = 0.95, eps, weight decay; "第 13 讲" §1.7: bias correction). */
typedef struct {
    float lr;
    float beta1;
    float beta2;
    float eps;
    float weight_decay;     /* used for BFO_FLAG_DECAY tensors; others use 0 */
    int32_t bias_correction;/* nonzero: divide m by 1 - beta1^t and v by 1 - beta2^t */
} bfo_adamw_hparams;

/* Output of grad_global_norm, written to device memory (16 bytes). */
typedef struct {
    double sumsq;  /* sum of squares of the shard's widened bf16 grads, binary64 */
    float norm;    /* (float)sqrt(sumsq) */
    float scale;   /* max_norm / norm if norm > max_norm, else 1 */
} bfo_norm_result;

/* Opaque handle: a validated tensor table intersected with one shard, plus
 * the small device-side lookup it needs (created once, reused every step). */
typedef struct bfo_table_s *bfo_table;

/* One run of a shard plan: shard-local elements [local, local + length) are
 * params/grads positions [addr, addr + length) and global indices
 * [global, global + length) of the flat buffer, all in one tensor-flag
 * class (flags bit 0 = decay).  addr equals local for FLAT tables and global
 * for PER_TENSOR tables.  Consecutive pieces with the same flag that continue
 * one another are merged into one run. */
typedef struct {
    uint64_t local;
    uint64_t addr;
    uint64_t global;
    uint64_t length;
    uint32_t flags;
    uint32_t reserved;
} bfo_run;

/* ZeRO-1 shard of an n-element buffer over `world` ranks
 * ("04 · 多 GPU 与混合精度" §3.2: shard = parameter count / process count,
 * which must divide exactly; "LLM 分布式训练实战" §3.1: rank r starts at
 * r * (n / world)).  Writes [*begin, *end) = [r*n/world, (r+1)*n/world).
 * Errors: BFO_EINVAL (world == 0 or null output), BFO_ERANGE (rank >= world),
 * BFO_ENOTDIVISIBLE (n % world != 0).  Host only; touches no GPU. */
int shard_range(uint64_t n, uint32_t world, uint32_t rank, uint64_t *begin, uint64_t *end);

/* Validates `tensors` (count entries, host memory, copied), takes rank
 * `rank`'s BFO_LAYOUT_FLAT shard of the buffer they describe and uploads the
 * shard plan to the current device.  Errors: as shard_range, BFO_ETABLE,
 * BFO_EINVAL (null out, or null tensors with count > 0), BFO_EHIP.  The
 * handle holds device memory until bfo_table_destroy. */
int bfo_table_create(const bfo_tensor *tensors, uint32_t count, uint32_t world, uint32_t rank,
                     bfo_table *out);

/* As bfo_table_create with an explicit layout (BFO_LAYOUT_FLAT or
 * BFO_LAYOUT_PER_TENSOR).  PER_TENSOR ("04 · 多 GPU 与混合精度" §3.2 and §6:
 * each tensor's size must divide by the process count) gives rank r
 * elements [offset + r*numel/N, offset + (r+1)*numel/N) of every tensor;
 * BFO_ENOTDIVISIBLE if any numel % world != 0.  Unknown layout: BFO_EINVAL. */
int bfo_table_create_layout(const bfo_tensor *tensors, uint32_t count, uint32_t world, uint32_t rank,
                            int layout, bfo_table *out);

/* Frees the handle and its device memory.  No call queued on the handle may
 * still be running.  NULL is accepted. */
int bfo_table_destroy(bfo_table table);

/* Buffer length n and the shard of a table: FLAT -> [begin, end); PER_TENSOR
 * -> begin = 0, end = S (the shard length). */
int bfo_table_info(bfo_table table, uint64_t *n, uint64_t *begin, uint64_t *end);

/* The table's shard plan: *count = number of runs; when out is not NULL,
 * copies them (BFO_ERANGE if capacity < *count).  Host only. */
int bfo_table_runs(bfo_table table, bfo_run *out, uint32_t capacity, uint32_t *count);

/* The shard plan bfo_table_create_layout would build, computed on the host
 * with no device and no table ("04 · 多 GPU 与混合精度" §3.2 for both layouts;
 * "LLM 分布式训练实战" §3.1 for the flat offset): the same validation and
 * status codes, *nruns = number of runs, *shard_elems (if not NULL) = S; when
 * out is not NULL, copies the runs (BFO_ERANGE if capacity < *nruns). */
int bfo_plan_runs(const bfo_tensor *tensors, uint32_t count, uint32_t world, uint32_t rank, int layout,
                  bfo_run *out, uint32_t capacity, uint32_t *nruns, uint64_t *shard_elems);

/* *bytes = the device workspace grad_global_norm needs for this table: one
 * binary64 partial per 8,192-element tile of the shard, plus one per 4,096
 * tiles above 32,768 tiles; 0 for shards of at most 8 tiles (65,536
 * elements), whose norm runs in one workgroup.  Host only. */
int bfo_norm_workspace_bytes(bfo_table table, uint64_t *bytes);

/* Deterministic global grad norm of one shard ("04 · 多 GPU 与混合精度" §4:
 * grad_norm, then grad_scale = min(1, 1/grad_norm), i.e. clip to 1.0; under
 * ZeRO-1 this is the shard's part, which ranks would add before the root).
 * grads: as in Arrays above.  out: device bfo_norm_result.  Every
 * square is formed and summed in binary64 over a fixed partition that
 * depends only on the shard length, so repeated calls give identical bits.
 * scale = max_norm / norm when norm > max_norm, else 1.0f (an infinite norm
 * gives 0, a NaN norm gives 1: non-finite grads are not sanitised, check
 * norm).  An empty shard gives {0, 0, 1}.  max_norm must be > 0 (+inf
 * turns clipping off); zero, negative or NaN -> BFO_EINVAL.
 * workspace: device memory of at least bfo_norm_workspace_bytes bytes,
 * 8-byte aligned, owned by the caller, written and read by this call only
 * (its contents before and after mean nothing); calls with separate
 * workspaces may run at the same time on different streams.  NULL uses a
 * buffer the table holds, so calls on one table with a NULL workspace must
 * not overlap in time. */
int grad_global_norm(bfo_table table, const uint16_t *grads, float max_norm, void *workspace,
                     bfo_norm_result *out, void *stream);

/* grad_global_norm for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same kernels, partition and bits, with the partials kept in
 * a fixed 8 MiB device array of the library instead of a workspace.  Every
 * GPU the library runs on holds its own copy of that array until the process
 * ends; its address is looked up on the first call on each device.  The call
 * allocates nothing.  Shards of up to 8,587,837,440 elements (1,048,320
 * norm tiles); larger ones -> BFO_ERANGE.  The array keeps the last call's
 * partials, which nothing reads (each call writes every partial it reads),
 * but all calls on one GPU share it: calls whose GPU work overlaps in time
 * on one GPU (different streams without ordering, or several threads) race
 * and give wrong norms.  Other arguments and errors as grad_global_norm. */
int grad_global_norm_noalloc(bfo_table table, const uint16_t *grads, float max_norm, bfo_norm_result *out,
                             void *stream);

/* One AdamW step over the shard ("04 · 多 GPU 与混合精度" §2.2, with the
 * lerp computed as two fused multiply-adds; "第 13 讲" §1.7 for bias
 * correction and decoupled decay).  Per element i (global) / j (local):
 *   g   = scale * f32(grads[j])
 *   m1  = fma(b1, m[j], fma(-b1, g, g));  v1 = fma(b2, v[j], fma(-b2, g*g, g*g))
 *   mh  = m1 / bc1;  vh = v1 / bc2;  u = mh / (sqrt(vh) + eps)
 *   old = master ? master[j] : f32(params[j])
 *   p   = old - lr * (u + w_i * old),  w_i = weight_decay if i's tensor has
 *         BFO_FLAG_DECAY else 0
 *   m[j] = m1; v[j] = v1; master[j] = p (when master != NULL);
 *   params[j] = SR(p, r16(i, seed)) or RNE(p)
 * each a single binary32 operation in that order.  bc1/bc2 =
 * (float)(1 - pow(beta, t)) in binary64, or 1 when bias correction is off.
 * SR rounds to the next bf16 away from zero when the 16 discarded bits of p
 * exceed r16, else truncates; r16 is a 16-bit draw of Philox4x32-10 (Salmon
 * et al., SC'11) with counter (lo32(i>>3), hi32(i>>3), 0, 0) and key
 * (lo32(seed), hi32(seed)); element i takes output word (i>>1)&3, low half
 * for even i.  RNE rounds to nearest, ties to even.  NaN stays NaN.
 * i is element j's global index (its run's global + offset), so every
 * layout and shard count draws the same r16 for the same parameter.
 * master == NULL selects the no-master path (old weights read from params).
 * scale: device float (e.g. &out->scale of grad_global_norm), or NULL for 1.
 * skip: device int32 (e.g. written by bfo_outlier_update), or NULL; when it
 * holds a nonzero value at run time the step changes nothing (every
 * workgroup exits after reading it).
 * t: 1-based step number (0 -> BFO_EINVAL).  rounding: BFO_ROUND_SR/RNE. */
int adamw_sr_step(bfo_table table, uint16_t *params, const uint16_t *grads, float *master, float *m,
                  float *v, const bfo_adamw_hparams *hp, const float *scale, const int32_t *skip, uint64_t t,
                  uint64_t seed, int rounding, void *stream);

/* grad_global_norm and then adamw_sr_step with that norm's clip scale, in
 * one call ("04 · 多 GPU 与混合精度" §4 for the norm and clip, §2.2 for the
 * update): the result -- *out, params, master, m, v -- is bit for bit that
 * of the two calls.  For shards of at most 65,536 elements (8 norm tiles)
 * both run in one kernel launch: every workgroup of the update forms the
 * whole shard's sum of squares itself, in the norm's partition and order,
 * so a small step pays one launch instead of two (workspace is then not
 * used); larger shards take the two calls' launches.  skip: as in
 * adamw_sr_step (the norm is still written).  Arguments and errors as the
 * two calls; out and workspace must not overlap the arrays. */
int adamw_sr_step_with_norm(bfo_table table, uint16_t *params, const uint16_t *grads, float *master, float *m,
                            float *v, const bfo_adamw_hparams *hp, float max_norm, void *workspace,
                            bfo_norm_result *out, const int32_t *skip, uint64_t t, uint64_t seed, int rounding,
                            void *stream);

/* The per-step scalars of adamw_sr_step, for a step whose launches are
 * recorded once (HIP graph capture) and replayed every step: they are read
 * from device memory when the step runs instead of being passed by value.
 * ("04 · 多 GPU 与混合精度" §4: the learning rate and the step number change
 * every step; "第 13 讲" §1.7: bias correction.)  32 bytes. */
typedef struct {
    float lr;
    float bc1;          /* 1 - beta1^t as adamw_sr_step forms it (1 when correction is off) */
    float bc2;          /* 1 - beta2^t, likewise */
    uint32_t reserved;  /* 0 */
    uint64_t t;         /* the 1-based step number these were formed for */
    uint64_t seed;      /* the step's rounding seed */
} bfo_step_scalars;

/* Host only: *out = the scalars adamw_sr_step(hp with lr, t, seed) uses --
 * bc1 and bc2 exactly as documented there.  hp->lr is ignored (lr is the
 * step's rate, e.g. from bfo_lr_at).  BFO_EINVAL for a null pointer or
 * t == 0. */
int bfo_step_scalars_fill(const bfo_adamw_hparams *hp, uint64_t t, float lr, uint64_t seed,
                          bfo_step_scalars *out);

/* adamw_sr_step with its per-step scalars taken on the device at run time:
 * the step uses steps[*cursor], where steps is a device array of `count`
 * bfo_step_scalars (16-byte aligned) and cursor a device uint64 (8-byte
 * aligned).  hp supplies beta1, beta2, eps and weight_decay; its lr and
 * bias_correction are ignored (the scalars carry them).  A cursor at or past
 * `count` makes the step change nothing, as a set skip flag does.  Every
 * other argument is as in adamw_sr_step, and for the same scalars the result
 * is the same bit for bit.  No argument varies from step to step, so a graph
 * recorded from grad_global_norm, this call and bfo_cursor_advance replays
 * step after step, the caller changing only the grads (and, if it likes,
 * the steps array) between replays. */
int adamw_sr_step_scheduled(bfo_table table, uint16_t *params, const uint16_t *grads, float *master, float *m,
                            float *v, const bfo_adamw_hparams *hp, const bfo_step_scalars *steps,
                            uint64_t count, const uint64_t *cursor, const float *scale, const int32_t *skip,
                            int rounding, void *stream);

/* *cursor += 1, on the device (one work-item), queued on stream. */
int bfo_cursor_advance(uint64_t *cursor, void *stream);

/* Resume-time rebuild ("04 · 多 GPU 与混合精度" §5.2): params at element j's
 * position = SR(master[j], r16(i, seed)) with the draws of adamw_sr_step, so
 * passing the seed of the update that produced `master` reproduces its
 * bf16 output bit for bit. */
int master_to_bf16_sr(bfo_table table, const float *master, uint16_t *params, uint64_t seed,
                      void *stream);

/* The same rebuild with a rounding mode: BFO_ROUND_SR as master_to_bf16_sr,
 * BFO_ROUND_RNE params = RNE(master[j]) (seed unused), which reproduces an
 * update made with round-to-nearest.  Unknown rounding: BFO_EINVAL. */
int master_to_bf16(bfo_table table, const float *master, uint16_t *params, uint64_t seed, int rounding,
                   void *stream);

/* Test export: out[k] = r16(first + k, seed) for k < count (device array,
 * 2-byte aligned).  Any first and count. */
int bfo_rng_dump(uint64_t first, uint64_t count, uint64_t seed, uint16_t *out, void *stream);

/* Test export: out[j] = 1 if shard element j's tensor has BFO_FLAG_DECAY,
 * else 0, as the update kernel sees it (device array of S bytes). */
int bfo_decay_mask_dump(bfo_table table, uint8_t *out, void *stream);

/* Measurement export: the update's memory traffic with none of its
 * arithmetic, for an achievable-bandwidth ceiling measured the same way as
 * the update, in the update's workgroup and lane plan (4-element quads:
 * 16-byte fp32 and 8-byte bf16 accesses) and with its cache policies.  For
 * j < count (device arrays of count elements):
 *   BFO_MIX_BOTH -- with a master: m[j], v[j], master[j] ^= key (as 32-bit
 *     patterns) and params[j] = grads[j] ^ (key & 0xFFFF): 14 bytes read and
 *     14 written per element, as the master update; master == NULL: m[j],
 *     v[j] ^= key and params[j] ^= grads[j] ^ (key & 0xFFFF): 12 read and 10
 *     written, as the no-master update.  key 0 leaves m, v and master
 *     unchanged;
 *   BFO_MIX_READS -- the same reads and no writes (14 or 12 bytes per
 *     element); nothing changes;
 *   BFO_MIX_WRITES -- the same writes and no reads (14 or 10 bytes per
 *     element) of words made from key and j: m, v, master and params are
 *     overwritten.
 * READS and WRITES time the two directions of the mix on their own.  Every
 * non-null pointer 16-byte aligned (else BFO_EMISALIGNED); unknown mode
 * BFO_EINVAL; count 0 is a no-op. */
enum { BFO_MIX_BOTH = 0, BFO_MIX_READS = 1, BFO_MIX_WRITES = 2 };
int bfo_stream_mix(uint16_t *params, const uint16_t *grads, float *master, float *m, float *v, uint64_t count,
                   uint32_t key, int mode, void *stream);

/* Learning-rate schedules ("04 · 多 GPU 与混合精度" §4 names cosine, linear,
 * constant and wsd; the formulas are this library's reading).  For 0-based
 * step s, lr_min = final_frac * lr_max, W = warmup_steps, T = total_steps:
 *   s < W: lr_max * (s + 1) / W (every kind);
 *   then, with p = min(1, (s - W) / (T - W)) (p = 1 when T == W):
 *   CONSTANT lr_max; LINEAR lr_max - (lr_max - lr_min) * p;
 *   COSINE lr_min + (lr_max - lr_min) * (1 + cos(pi * p)) / 2;
 *   WSD lr_max until s >= T - D with D = decay_frac * T, then linear from
 *   lr_max to lr_min over those last D steps.
 * Evaluated in binary64, rounded once to binary32.  Host only. */
enum { BFO_LR_CONSTANT = 0, BFO_LR_LINEAR = 1, BFO_LR_COSINE = 2, BFO_LR_WSD = 3 };
typedef struct {
    int32_t kind;
    uint32_t reserved;
    uint64_t warmup_steps;
    uint64_t total_steps;   /* >= warmup_steps */
    float lr_max;
    float final_frac;
    float decay_frac;       /* WSD only */
    uint32_t reserved2;
} bfo_lr_schedule;

/* *lr = the schedule's learning rate at step `step`.  BFO_EINVAL for a null
 * argument, an unknown kind or total_steps < warmup_steps. */
int bfo_lr_at(const bfo_lr_schedule *schedule, uint64_t step, float *lr);

/* Outlier detector ("04 · 多 GPU 与混合精度" §4: z-score of the grad norm
 * over a window of 128 values; the update is skipped when it exceeds a
 * threshold).  State lives in device memory so the decision never leaves
 * the GPU.  bfo_outlier_update reads *value (device float, e.g.
 * &norm_out->norm), and writes, on `stream`:
 *   *z    = (value - mean) / sqrt(variance) of the previous `window` finite
 *           values (binary64, population variance, summed oldest to newest),
 *           NaN until `window` values have been seen;
 *   *skip = 1 if value is not finite, or threshold > 0 and z > threshold;
 *           else 0 (pass skip to adamw_sr_step);
 * then appends value to the window if it is finite.  window: 1..4096. */
typedef struct bfo_outlier_s *bfo_outlier;
int bfo_outlier_create(uint32_t window, float threshold, bfo_outlier *out);
int bfo_outlier_destroy(bfo_outlier detector);
/* Empties the window (queued on `stream`). */
int bfo_outlier_reset(bfo_outlier detector, void *stream);
int bfo_outlier_update(bfo_outlier detector, const float *value, float *z, int32_t *skip, void *stream);

/* Checkpoints ("04 · 多 GPU 与混合精度" §5.1-5.2).  Each rank saves its own
 * optimizer state; a DONE marker written after every rank has saved makes
 * the checkpoint count; resume takes the newest step with a marker.  With a
 * master, the bf16 weights need not be saved: loading rebuilds them from the
 * master with the saved seed and rounding mode, bit-identical to the ones
 * the saved step produced, and because only the master is needed the same
 * state can also resume a run without a master (the page's precision switch
 * at resume).
 *
 * bfo_checkpoint_save writes <dir>/state_<step:08>_<rank:05>.bin: a 128-byte
 * header (magic "BFOSTATE", version 2, step, seed, n, S, world, rank,
 * layout, whether a master and whether params are stored, a fingerprint of
 * the tensor table, the rounding mode, a checksum of each payload array and
 * one of the header) and the payload: master (S fp32) when master is not
 * NULL, the shard's bf16 params in shard-local order when params is not NULL
 * (params addressed as in adamw_sr_step), then m and v (S fp32 each).  At
 * least one of master and params must be given.  step is the last step the
 * state includes; seed and rounding (BFO_ROUND_SR / BFO_ROUND_RNE) are those
 * of the last update that changed the state.  Pass params too when that
 * update is not known for sure -- e.g. when a device skip flag may have
 * dropped it: the stored params are then restored as they are.  The
 * checksums are bfo_checksum64 of each array's bytes as stored.  Device
 * arrays are copied through a pinned buffer on `stream` after the work
 * already queued there; the call returns when the file is on disk (written
 * under a temporary name, synced, renamed into place, directory synced).
 * Errors: BFO_EINVAL, BFO_EIO, BFO_EHIP. */
int bfo_checkpoint_save(const char *dir, bfo_table table, const uint16_t *params, const float *master,
                        const float *m, const float *v, uint64_t step, uint64_t seed, int rounding, void *stream);

/* Creates the empty marker <dir>/DONE_<step:08> and syncs it and the
 * directory to disk. */
int bfo_checkpoint_done(const char *dir, uint64_t step);

/* *step = the largest step with a DONE marker in dir; BFO_ENOTFOUND if none. */
int bfo_checkpoint_latest(const char *dir, uint64_t *step);

/* Reads this rank's state of `step`; *seed (if not NULL) gets the saved seed.
 * m and v are always read.  master not NULL: the stored master is read into
 * it (BFO_EFORMAT if the file has none).  params not NULL: the shard's
 * positions of params get the stored params if the file has them, else they
 * are rebuilt from the stored master as master_to_bf16 does with the saved
 * seed and rounding mode -- also when master is NULL, which resumes a
 * master checkpoint in a run without one (v's buffer then holds the master
 * while the params are rebuilt, before v is read).  master and params may
 * not both be NULL.  BFO_ENOTFOUND if the file is missing; BFO_EFORMAT if
 * its header does not match the table (sizes, world, rank, layout,
 * fingerprint), the file is truncated, or a checksum does not match (the
 * arrays then hold partly loaded data and must not be used). */
int bfo_checkpoint_load(const char *dir, uint64_t step, bfo_table table, uint16_t *params, float *master,
                        float *m, float *v, uint64_t *seed, void *stream);

/* The 64-bit checksum stored in checkpoint headers, of `bytes` bytes of host
 * memory: four lanes h[0..3] (h[l] starting at the 64-bit FNV-1a offset
 * basis + l) take the data in 32-byte blocks (the last one padded with
 * zeros), lane l folding the block's l-th little-endian 8-byte word w in as
 * h[l] = (h[l] ^ w) * 1099511628211; then x = basis ^ bytes and, for each
 * lane in order, x = (x ^ h[l]) * 1099511628211, x ^= x >> 29.  A change
 * that stays within one 8-byte word always changes the result.  Host only. */
uint64_t bfo_checksum64(const void *data, uint64_t bytes);

/* Placement of the step's arrays in device memory (a measured property of
 * MI355X, not of the method).  The update streams five arrays at the same
 * element index -- params, grads, master, m, v -- and it moves its bytes
 * about 15% faster (6.1 against 5.3 TB/s on the 1.5B model's shard) when
 * every pair of them lies in different 16 GiB-aligned regions of physical
 * device memory, i.e. their physical addresses differ in bit 34 or above;
 * sharing a region, even at gigabytes' distance, gives the lower rate.  The
 * library does not allocate these arrays; a caller can get the placement by
 * carving them from one allocation that covers most of the device (whose
 * physical backing then follows its virtual layout) at the offsets below,
 * and fill the gaps with its other buffers.  Placement changes no result.
 *
 * Which regions also matters, a little for five arrays and a lot for four:
 * four arrays in the four regions of one 64 GiB-aligned block run at the
 * lower rate again, so the layout below starts no array in the fourth
 * region of a block.
 *
 * bfo_spread_layout: for `count` arrays of bytes[k] bytes (in that order),
 * offsets[k] = the first multiple of BFO_REGION_BYTES at or after the end
 * of array k-1 that is not the fourth region of a 64 GiB-aligned block
 * (offsets[0] = 0); *total = offsets[count-1] + bytes[count-1] (0 when
 * count is 0).  BFO_EINVAL for null pointers with count > 0 and BFO_ERANGE
 * if an offset or the total does not fit in 64 bits.  Host only. */
#define BFO_REGION_BYTES (1ull << 34)
int bfo_spread_layout(const uint64_t *bytes, uint32_t count, uint64_t *offsets, uint64_t *total);

/* ---------------------------------------------------------------------------
 * Operators of the training loop around the step: where the grads come from.
 *
 * Layer norm, the log probabilities of given tokens and distillation from a
 * teacher's top logits, each with its gradient.  They take no table: every
 * array is a plain device array on the current device.  Conventions beside
 * those at the top of this file:
 *   - Matrices are row-major with unit column stride; a `stride` is the
 *     distance between rows in elements, at least the row's width (rows of a
 *     wider buffer, or columns of one, are fine).  Rows and matrices may start
 *     anywhere their type allows (2 bytes for bf16, 4 for fp32).
 *   - dtype / param_dtype: BFO_BF16 (bf16 patterns) or BFO_F32; anything else
 *     BFO_EINVAL.  All arithmetic is binary32; an output in bf16 is rounded
 *     once, to nearest even.
 *   - rows may be 0 (the matrices may then be NULL).
 *   - Results are the same bits from call to call on the same arrays: sums run
 *     in an order that depends on the sizes only, and there are no atomics in
 *     them.  In the forward passes over a vocabulary the order depends also on
 *     where in a 128-byte line of memory each row starts, so that the same scores
 *     at another start (or as another row of an odd stride) may differ within
 *     binary32 rounding; top_index and the gradients of given stats do not.
 *   - Outputs may not overlap an input or one another, except where a call
 *     says so (BFO_EINVAL).  Only the rows' own elements are written.
 *   - Workspaces are device memory, 16-byte aligned, of the size the matching
 *     *_workspace_bytes gives for the call's sizes or larger ones (it never falls
 *     as one of them grows), owned by the caller and used by this call only;
 *     calls with separate workspaces may run at the same time, and graphs that
 *     may run at the same time need a workspace each.  Calls allocate nothing
 *     and can be recorded into a HIP graph.
 *   - Errors: BFO_EINVAL, BFO_EMISALIGNED, BFO_ERANGE (a size or stride above
 *     its limit), BFO_EHIP.
 * ------------------------------------------------------------------------- */
enum { BFO_BF16 = 0, BFO_F32 = 1 };

/* Layer norm over the columns of x (rows x cols).  Per row:
 *   mean = sum(x) / cols;  rstd = 1 / sqrt(sum((x - mean)^2) / cols + eps)
 *   out = (x - mean) * rstd * weight + bias
 * weight and bias hold cols values of param_dtype; bias may be NULL (0).
 * out has x's type.  mean and rstd (rows floats each, for the backward pass)
 * may be NULL.  1 <= cols <= BFO_LAYERNORM_MAX_COLS (0 -> BFO_EINVAL, above ->
 * BFO_ERANGE); eps >= 0 and finite.  A row with an infinity or NaN gives NaN.
 * The sums are binary32's, which holds them for |x| < 2^113 and differences from
 * the mean below 2^56; a row beyond that overflows (a sum of squares that does
 * gives rstd 0 and out = bias).  Where eps = 0, a row whose differences are all
 * below 2^-56 may lose their squares, and a constant row has no finite result. */
#define BFO_LAYERNORM_MAX_COLS 16384u
int layernorm_forward(const void *x, uint64_t x_stride, const void *weight, const void *bias, void *out,
                      uint64_t out_stride, float *mean, float *rstd, uint64_t rows, uint32_t cols, float eps,
                      int dtype, int param_dtype, void *stream);

/* *bytes = the workspace layernorm_backward needs; 0 for few rows (up to
 * 2,048 of at most 2,048 columns, 1,024 of at most 4,096, 512 of more), and
 * workspace may then be NULL.  Host only. */
int bfo_layernorm_workspace_bytes(uint64_t rows, uint32_t cols, uint64_t *bytes);

/* Gradients of layernorm_forward, from its mean and rstd.  With
 * xhat = (x - mean) * rstd and h = weight * dout, per row:
 *   dx = rstd * (h - sum(h) / cols - xhat * sum(h * xhat) / cols)
 * and over the rows dweight = sum(dout * xhat), dbias = sum(dout).
 * dout and dx have x's type, dweight and dbias param_dtype (so they can be the
 * layer's places in the flat grads buffer); dbias may be NULL.
 * accumulate: 0, or BFO_ACCUMULATE_DX (dx += , the residual stream's gradient)
 * and/or BFO_ACCUMULATE_PARAMS (dweight, dbias += , micro-batches); the sum is
 * formed in binary32 and rounded once.  rows == 0 writes (or adds) zeros to
 * dweight and dbias. */
enum { BFO_ACCUMULATE_DX = 1, BFO_ACCUMULATE_PARAMS = 2 };
int layernorm_backward(const void *dout, uint64_t dout_stride, const void *x, uint64_t x_stride,
                       const void *weight, const float *mean, const float *rstd, void *dx, uint64_t dx_stride,
                       void *dweight, void *dbias, uint64_t rows, uint32_t cols, int dtype, int param_dtype,
                       int accumulate, void *workspace, void *stream);

/* *bytes = the workspace of token_logprobs_forward (top tokens asked for) and
 * distill_forward (top 0), which calls of up to 128 rows of at least 65,536
 * scores need; to others workspace may be NULL.  Host only. */
int bfo_logits_workspace_bytes(uint64_t rows, uint32_t vocab, uint32_t top, uint64_t *bytes);

/* Log probabilities of given tokens.  Row r of logits holds vocab scores (a
 * wider row's further columns are not read); with z = scale * logits (scale:
 * 1 / temperature, finite and > 0), M = max(z), S = sum(exp(z - M)):
 *   stats[r] = {M, log(S)}  (2 floats; log-sum-exp = M + log(S))
 *   logprob[r] = z[targets[r]] - M - log(S)
 *   entropy[r] = log(S) - sum(exp(z - M) * (z - M)) / S
 *   top_index[r][k], top_logprob[r][k], k < top: the `top` largest logits,
 *     largest first, equal ones by the lower index, and their log probabilities.
 * targets, logprob (both or neither), stats and entropy may be NULL;
 * top <= BFO_TOP_MAX and <= vocab; top == 0 takes neither top array.
 * A negative target masks its row: logprob 0.  A target >= vocab is no token:
 * logprob NaN.  Scores of -inf have probability 0; a row of nothing else has
 * stats {-inf, 0}, entropy 0 and log probabilities -inf.  (Scores count as
 * infinite where z overflows binary32.)  A row with a NaN or
 * +inf has NaN stats, entropy and log probabilities (top_index then orders NaN
 * first).  1 <= vocab <= BFO_VOCAB_MAX. */
#define BFO_TOP_MAX 128u
#define BFO_VOCAB_MAX (1u << 28)
int token_logprobs_forward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, int dtype,
                           float scale, const int32_t *targets, float *logprob, float *stats, float *entropy,
                           uint32_t top, int32_t *top_index, float *top_logprob, void *workspace, void *stream);

/* Gradient of sum(dlogprob * logprob + dentropy * entropy) with respect to the
 * logits, from the forward pass's stats and entropy.  With p = exp(z - M - log S),
 * z rounded to binary32 first:
 *   dlogits[j] = scale * (dlogprob * ([j == target] - p[j])
 *                         - dentropy * p[j] * (log p[j] + entropy))   j < vocab
 *   dlogits[j] = 0                                                    vocab <= j < width
 * (cross entropy: dlogprob = -1 / tokens.)  dlogits: rows of width >= vocab
 * columns, of the logits' type; it may be the logits themselves (same pointer
 * and stride).  targets and dlogprob, entropy and dentropy: both or neither of
 * a pair, at least one pair.  Rows whose factors are all 0 (masked targets
 * count as 0) and rows of -inf only get exact zeros, whatever they hold; a
 * target >= vocab gives a row of NaN. */
int token_logprobs_backward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, uint32_t width,
                            int dtype, float scale, const int32_t *targets, const float *stats,
                            const float *entropy, const float *dlogprob, const float *dentropy, void *dlogits,
                            uint64_t dlogits_stride, void *stream);

/* Distillation loss against a teacher's top logits.  Row r names `count`
 * teacher tokens (teacher_index, teacher_logits: rows x count, contiguous; a
 * negative index is no entry).  With q = softmax(scale * teacher_logits) over
 * the row's entries and p the student's probabilities over the whole
 * vocabulary, as in token_logprobs_forward:
 *   kl[r] = sum_k q[k] * (log q[k] - log p[teacher_index[k]])
 * (0 for a row without entries, or with entries of -inf only; an entry of
 * probability 0 adds nothing).  One scale
 * serves the teacher, the student and the true tokens' logprob.  Any per-row
 * constant in the teacher's logits drops out, so top_logprob of the teacher's
 * token_logprobs_forward serves too if that ran at scale 1; at another scale s it
 * holds scaled scores, and q would be softmax(scale * s * logits): such a caller
 * takes the scores themselves, logits[r][top_index[r][k]], or top_logprob / s.
 * A token named twice counts with
 * both probabilities.  An index >= vocab, or a NaN or +inf among the entries,
 * gives NaN.  stats, targets and logprob as in token_logprobs_forward (all may
 * be NULL), so that a loss on the true tokens takes no second pass.
 * 1 <= count <= BFO_TOP_MAX. */
int distill_forward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, int dtype, float scale,
                    const int32_t *teacher_index, const float *teacher_logits, uint32_t count,
                    const int32_t *targets, float *kl, float *logprob, float *stats, void *workspace,
                    void *stream);

/* Gradient of sum(dkl * kl + dlogprob * logprob) with respect to the student's
 * logits (the teacher gets none):
 *   dlogits[j] = scale * (dkl * (p[j] - q[j]) + dlogprob * ([j == target] - p[j]))
 * with q[j] the sum over the entries naming j, and dkl counted as 0 in a row
 * without entries.  targets and dlogprob: both or neither.  dlogits, width,
 * zero and NaN rows as in token_logprobs_backward. */
int distill_backward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, uint32_t width,
                     int dtype, float scale, const int32_t *teacher_index, const float *teacher_logits,
                     uint32_t count, const int32_t *targets, const float *stats, const float *dkl,
                     const float *dlogprob, void *dlogits, uint64_t dlogits_stride, void *stream);

/* ---------------------------------------------------------------------------
 * Operators between a transformer block's matrix products: root-mean-square
 * norm with the residual's addition, the feed-forward's activation, rotary
 * positions, each with its gradient, and what a training step keeps between
 * forward and backward in 8 bits.  Conventions as above.
 *
 * Codes.  rows x cols values are kept as one byte each (codes: a matrix of
 * bytes, rows `codes_stride` bytes apart, starting anywhere) and a binary32
 * scale for every group of BFO_GROUP columns of a row (scales: rows x
 * ceil(cols / BFO_GROUP), contiguous; the last group of a row may be shorter),
 * or, where a call takes group == 0, one scale for the whole row (scales: rows).
 * With amax the group's largest absolute value and top = 127 (BFO_I8: signed
 * integers) or 448 (BFO_E4M3: 8-bit floats of 4 exponent and 3 mantissa bits,
 * no infinities), in binary32
 *   scale = max(amax * (1 / top), 2^-126)
 *   code  = value * (1 / scale), rounded to the nearest code, ties to even
 * and a code stands for code * scale: at most scale / 2 off for integers, a
 * 16th of itself (or scale * 2^-10, if more) for e4m3.  A group with a NaN or
 * an infinity stands for NaN throughout.
 * ------------------------------------------------------------------------- */
enum { BFO_I8 = 0, BFO_E4M3 = 1 };
#define BFO_GROUP 128u

/* Root-mean-square norm of x + residual.  Per row:
 *   total = x + residual, rounded to the type (x itself where residual is NULL)
 *   rstd = 1 / sqrt(sum(total^2) / cols + eps)
 *   normalised = total * rstd;  out = normalised * weight
 * weight holds cols values of param_dtype.  total, out and rstd (rows floats,
 * for the backward pass) may be NULL, total must be without a residual; total
 * may be x or residual (same pointer and stride).  codes and scales, both or
 * neither: codes_of BFO_CODES_OF_OUT keeps out (for a product in 8 bits; out
 * before its rounding), BFO_CODES_OF_NORMALISED the normalised row (for the
 * backward pass); group BFO_GROUP or 0.  At least one of out and codes must be
 * given.  1 <= cols <= BFO_RMSNORM_MAX_COLS (0 -> BFO_EINVAL, above ->
 * BFO_ERANGE); eps >= 0 and finite.  A row with a NaN gives NaN, one with an
 * infinity rstd 0 and NaN in its place.  The sum of squares is binary32's, which
 * holds it for |total| < 2^57 (beyond, it may overflow: rstd 0 and out 0); where
 * eps = 0, a row of zeros has no finite result, and one below 2^-56 may lose its
 * squares. */
#define BFO_RMSNORM_MAX_COLS 16384u
enum { BFO_CODES_OF_OUT = 0, BFO_CODES_OF_NORMALISED = 1 };
int rmsnorm_forward(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride,
                    const void *weight, void *total, uint64_t total_stride, void *out, uint64_t out_stride,
                    float *rstd, void *codes, uint64_t codes_stride, float *scales, int code_type, int codes_of,
                    uint32_t group, uint64_t rows, uint32_t cols, float eps, int dtype, int param_dtype,
                    void *stream);

/* *bytes = the workspace rmsnorm_backward needs; 0 for few rows (up to 2,048 of
 * at most 2,048 columns, 1,024 of at most 4,096, 512 of at most 8,192, 256 of
 * more), and workspace may then be NULL.  Host only. */
int bfo_rmsnorm_workspace_bytes(uint64_t rows, uint32_t cols, uint64_t *bytes);

/* Gradients of rmsnorm_forward, from its rstd and either the row that it
 * normalised (x: the forward pass's total) or that row's codes of
 * BFO_CODES_OF_NORMALISED (x NULL).  With xhat = x * rstd, or what the codes
 * stand for, and h = weight * dout, per row:
 *   dx = rstd * (h - xhat * sum(h * xhat) / cols)
 * (the gradient of x, of the residual and of total alike), and over the rows
 * dweight = sum(dout * xhat).  out, unless NULL, gets xhat * weight again, which
 * the next product's weight gradient needs and a step that keeps codes has not
 * kept.  accumulate, rows == 0 and the types as in layernorm_backward. */
int rmsnorm_backward(const void *dout, uint64_t dout_stride, const void *x, uint64_t x_stride, const void *codes,
                     uint64_t codes_stride, const float *scales, int code_type, uint32_t group, const void *weight,
                     const float *rstd, void *dx, uint64_t dx_stride, void *dweight, void *out, uint64_t out_stride,
                     uint64_t rows, uint32_t cols, int dtype, int param_dtype, int accumulate, void *workspace,
                     void *stream);

/* The feed-forward's activation: out = act(gate) * up, or act(gate) where up is
 * NULL, with act(g) = g / (1 + exp(-z)) and
 *   BFO_SILU  z = g
 *   BFO_GELU  z = 2 sqrt(2 / pi) (g + 0.044715 g^3)   (GELU's tanh form)
 * gate_codes with gate_scales, and up_codes with up_scales where up is given,
 * keep both inputs in codes for the backward pass (all of them or none), in
 * groups of BFO_GROUP columns.  out may be gate or up (same pointer and stride).
 * NaN and infinities in gate give what the formula does (-inf: NaN).
 * 1 <= cols <= BFO_ACTIVATION_MAX_COLS; rows * ceil(cols / BFO_GROUP) <= 2^31
 * (above -> BFO_ERANGE). */
enum { BFO_SILU = 0, BFO_GELU = 1 };
#define BFO_ACTIVATION_MAX_COLS (1u << 28)
int activation_forward(const void *gate, uint64_t gate_stride, const void *up, uint64_t up_stride, void *out,
                       uint64_t out_stride, void *gate_codes, uint64_t gate_codes_stride, float *gate_scales,
                       void *up_codes, uint64_t up_codes_stride, float *up_scales, int code_type, uint64_t rows,
                       uint32_t cols, int kind, int dtype, void *stream);

/* Gradients of activation_forward at its inputs (gate, and up if it was given)
 * or at what their codes stand for (gate and up NULL):
 *   dgate = dout * up * act'(gate);  dup = dout * act(gate)
 * (without up: dgate = dout * act'(gate), and dup is NULL).  out, unless NULL,
 * gets act(gate) * up again, for the next product's weight gradient.  Each
 * output may be one of dout, gate and up (same pointer and stride), none the
 * codes. */
int activation_backward(const void *dout, uint64_t dout_stride, const void *gate, uint64_t gate_stride,
                        const void *up, uint64_t up_stride, const void *gate_codes, uint64_t gate_codes_stride,
                        const float *gate_scales, const void *up_codes, uint64_t up_codes_stride,
                        const float *up_scales, int code_type, void *dgate, uint64_t dgate_stride, void *dup,
                        uint64_t dup_stride, void *out, uint64_t out_stride, uint64_t rows, uint32_t cols, int kind,
                        int dtype, void *stream);

/* Any other activation that a step keeps in 8 bits: its codes in groups of
 * BFO_GROUP columns, and the values that codes (of either group) stand for, in
 * binary32 or rounded to bf16.  Sizes as in activation_forward. */
int activation_pack(const void *x, uint64_t x_stride, void *codes, uint64_t codes_stride, float *scales,
                    int code_type, uint64_t rows, uint32_t cols, int dtype, void *stream);
int activation_unpack(const void *codes, uint64_t codes_stride, const float *scales, int code_type, uint32_t group,
                      void *out, uint64_t out_stride, uint64_t rows, uint32_t cols, int dtype, void *stream);

/* The angle per position of each pair of a head's rotated columns, with base >
 * 1: frequency[i] = base^(-2 i / rotated), i < rotated / 2, and for contexts
 * `factor` >= 1 times as long as the `length` positions that a model was
 * trained on:
 *   BFO_ROTARY_UNSCALED  as it is
 *   BFO_ROTARY_LINEAR    divided by factor
 *   BFO_ROTARY_BASE      of the base * factor^(rotated / (rotated - 2)): the first
 *                        as it is, the last divided by factor (rotated >= 4)
 *   BFO_ROTARY_BY_TURNS  divided by factor below `low` turns in length positions,
 *                        as it is above `high`, and between them mixed in proportion
 *                        to the number of turns
 *   BFO_ROTARY_BY_PAIR   the same, mixed in proportion to the pair's index, between
 *                        the (real) indexes that make these turns; a model whose
 *                        bounds were rounded to whole pairs brings its own frequencies
 * (0 < low < high; length and these two are used by the last two kinds only).
 * frequencies: rotated / 2 doubles of host memory, which a caller copies to the
 * device once.  rotated: even, 2 ... BFO_ROTARY_MAX_DIM.  BFO_EINVAL for
 * anything else.  Host only. */
#define BFO_ROTARY_MAX_DIM 1024u
#define BFO_ROTARY_MAX_HEADS 65535u
enum {
    BFO_ROTARY_UNSCALED = 0,
    BFO_ROTARY_LINEAR = 1,
    BFO_ROTARY_BASE = 2,
    BFO_ROTARY_BY_TURNS = 3,
    BFO_ROTARY_BY_PAIR = 4
};
typedef struct {
    int32_t kind;
    uint32_t reserved;  /* not read */
    double base;
    double factor;
    double length;
    double low;
    double high;
} bfo_rotary_scaling;
int bfo_rotary_frequencies(const bfo_rotary_scaling *scaling, uint32_t rotated, double *frequencies);

/* Rotary positions: out = x with the pairs of every head's first `rotated`
 * columns turned by the token's position times the pair's frequency:
 *   (a, b) -> amplitude * (a cos - b sin, a sin + b cos)
 * Pair i is columns (i, i + rotated / 2) for BFO_ROTARY_HALF, (2 i, 2 i + 1) for
 * BFO_ROTARY_INTERLEAVED.  Columns from rotated on are copied.  backward != 0
 * turns back (b's signs change places): x is then the gradient of the turned
 * heads and out that of the heads before.
 * x, out: head h of token t starts at t * token_stride + h * head_stride and
 * holds head_dim values with unit stride; either the tokens' rows or the heads'
 * may be the outer ones, but they may not reach into one another (so queries and
 * keys of one buffer take one call).  out may be x (same pointer and strides);
 * the columns behind are then not touched.
 * frequencies: device array of rotated / 2 doubles (8-byte aligned), in radians
 * per position.  positions: device array of tokens int32 (any sign), or NULL:
 * position t, or t % period where period is not 0 (sequences of that length, one
 * after the other).  Angles are formed and reduced in binary64, the rest is
 * binary32, rounded once.  amplitude (finite): 1, or what a long context's
 * scaling asks for.  heads <= BFO_ROTARY_MAX_HEADS, head_dim <=
 * BFO_ROTARY_MAX_DIM, rotated even, 2 ... head_dim. */
enum { BFO_ROTARY_HALF = 0, BFO_ROTARY_INTERLEAVED = 1 };
int rotary_apply(const void *x, uint64_t x_token_stride, uint64_t x_head_stride, void *out,
                 uint64_t out_token_stride, uint64_t out_head_stride, uint64_t tokens, uint32_t heads,
                 uint32_t head_dim, uint32_t rotated, int layout, const double *frequencies,
                 const int32_t *positions, uint64_t period, float amplitude, int backward, int dtype, void *stream);

/* Static string naming a status code. */
const char *bfo_status_string(int status);

/* hipError_t code of the last HIP failure seen by the calling thread (0 if none). */
int bfo_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* BF16OPT_H */
