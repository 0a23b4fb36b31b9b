/*
 * shardstate.h -- C ABI of the GB300 (sm_103a) sharded-state step of FSDP /
 * ZeRO-3 data parallelism, with N virtual data-parallel ranks held as N
 * buffers in one GPU's HBM.
 *
 * One training step of a fully sharded data-parallel group, as the pages
 * describe it ("Scaling data parallel", sections 9.1-9.3; "FSDP1 vs FSDP2",
 * sections 03-04; "ai-infra-kb M036", section 04 layer lifecycle):
 *   1. every rank's gradient is laid out in the group's sharded layout
 *      (fsdp_pack);
 *   2. a reduce-scatter leaves rank s the mean over ranks of its 1/N shard,
 *      and each rank runs mixed-precision AdamW on its own shard of the fp32
 *      master weights and moments, writing its bf16 parameter shard
 *      (fsdp_reduce_scatter_adamw, one fused pass);
 *   3. an all-gather returns the full parameters, read back out per
 *      parameter (fsdp_all_gather_unpack).
 * DDP's bucketed gradient all-reduce sits beside it
 * (ddp_bucket_pack_average), and so do the loss at the head of the model
 * (ss_linear_cross_entropy) and the global gradient norm with clipping
 * (ss_clip_grads; fsdp_reduce_scatter_norm and fsdp_clip_adamw for the
 * sharded step).
 *
 * Conventions for every call:
 *   - Status: 0 (SS_OK) or a negative SS_E* code; ss_strerror() names it.
 *     Argument errors are detected on the host before anything is launched.
 *     SS_ECUDA means a CUDA runtime call failed; ss_last_cuda_error() returns
 *     that cudaError_t value for the calling thread.
 *   - Device pointers are plain device addresses on the current CUDA device.
 *     A plan's metadata lives on the device that was current when it was
 *     created; launching calls made with another device current return
 *     SS_EINVAL.
 *     The caller owns all of them; the library never frees or keeps them.
 *   - Launches are asynchronous on the caller's stream (NULL = the legacy
 *     default stream).  Nothing synchronises except plan creation, which
 *     copies the plan's metadata to the device before it returns.
 *   - Pointer arrays (params, rank_grads, params_out, avg_out) are HOST
 *     arrays of device pointers; they are read during the call and may be
 *     reused as soon as it returns.
 *   - The arithmetic never traps: no device-side assert, no trap, and no
 *     kernel waits on another.  Waits inside a kernel (for copies, products, the
 *     other CTAs of a cluster, and in ss_clip_grads and ss_grad_norm the grid of a
 *     cooperative launch) are bounded or end with the CTAs themselves.
 *
 * Element types: elem_bytes 2 = bf16 (gradients, parameters, shards),
 * elem_bytes 4 = fp32.  Optimizer state is always fp32.
 */
#ifndef SHARDSTATE_H
#define SHARDSTATE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without pulling in the CUDA headers. */
typedef struct CUstream_st* ss_stream_t;

enum {
    SS_OK = 0,
    SS_EINVAL = -1,    /* bad argument: null pointer, size, world size, dtype, index */
    SS_EALIGN = -2,    /* pointer not aligned as the call requires */
    SS_EOVERFLOW = -3, /* a size overflows int64 / the index types */
    SS_ENOMEM = -4,    /* host or device allocation failed */
    SS_ECUDA = -5,     /* a CUDA runtime call failed (ss_last_cuda_error) */
    SS_ENODEVICE = -6, /* the plan has no device metadata (created host-only) */
    SS_ESCRATCH = -7   /* the call needs more than the library's fixed scratch array */
};

/* Largest N (virtual ranks) the kernels accept. */
#define SS_MAX_WORLD 64
/* Largest number of output replicas fsdp_all_gather_unpack writes per call. */
#define SS_MAX_REPLICAS 64

/*
 * Sharded layouts ("FSDP1 vs FSDP2", section 03, and its 3+5-element table).
 *  SS_FLAT_ORIG_FALSE  FSDP1 FlatParameter, use_orig_params=False (default):
 *                      plain concatenation (length L), torch.chunk(N), every
 *                      rank padded to c = ceil(L/N).
 *  SS_FLAT_ORIG_TRUE   FSDP1 FlatParameter, use_orig_params=True: from the
 *                      2nd parameter on, zero padding so it starts on a 16-byte
 *                      boundary (at most 16/elem_bytes - 1 elements), then the
 *                      buffer padded to a multiple of N; c = padded length / N.
 *  SS_PER_PARAM_DIM0   FSDP2 per-parameter DTensor(Shard(0)): parameter i is
 *                      split on dim 0 into chunks of c_i = ceil(d0_i/N) rows
 *                      (an empty parameter gives empty chunks); rank r's shard
 *                      concatenates its (padded) chunk of every parameter of
 *                      the group, S = sum_i c_i * inner_i.
 */
typedef enum {
    SS_FLAT_ORIG_FALSE = 0,
    SS_FLAT_ORIG_TRUE = 1,
    SS_PER_PARAM_DIM0 = 2
} ss_layout;

/* Opaque plan: layout metadata on the host plus its device copy. */
typedef struct ss_plan ss_plan;

/* Plan creation flag: compute the layout on the host only (no device
 * allocation or copy).  Such a plan answers the query calls; launching calls
 * return SS_ENODEVICE. */
#define SS_PLAN_HOST_ONLY 1u

/*
 * Description of a plan.  Parameters are numbered 0..num_params-1 in
 * registration order; parameter i has shape (dim0[i], inner[i]) where inner
 * is the product of the trailing dims (inner == NULL means 1 for all;
 * a 0-d parameter is (1, 1)).  Consecutive parameters form fully_shard groups
 * ("FSDP1 vs FSDP2", section 04: sharding unit = parameter, communication
 * unit = group): group g holds group_num_params[g] parameters.  num_groups 0
 * or group_num_params NULL means one group holding every parameter.  For the
 * FLAT layouts each group is one FlatParameter.
 */
typedef struct {
    ss_layout kind;
    int world_size;                /* N, 1..SS_MAX_WORLD */
    int elem_bytes;                /* 2 (bf16) or 4 (fp32) */
    int num_params;                /* >= 0 */
    const int64_t* dim0;           /* [num_params], each >= 0 */
    const int64_t* inner;          /* [num_params] or NULL, each >= 0 */
    int num_groups;                /* 0 = one group */
    const int* group_num_params;   /* [num_groups], summing to num_params */
    unsigned flags;                /* SS_PLAN_HOST_ONLY or 0 */
} ss_plan_desc;

/*
 * Packed-buffer geometry.  Every packed buffer of a plan (each rank's
 * gradients, the optimizer state, the parameter shards) has total_numel
 * elements.  Group g occupies [base_g, base_g + N*S_g); inside it rank r's
 * shard is [base_g + r*S_g, base_g + (r+1)*S_g).  For the FLAT layouts the N
 * shards of a group side by side are exactly the padded FlatParameter.
 */
typedef struct {
    int64_t shard_numel;     /* elements per rank, summed over groups */
    int64_t total_numel;     /* N * shard_numel */
    int64_t unpadded_numel;  /* sum of parameter numels */
    int64_t pad_numel;       /* total_numel - unpadded_numel */
    int world_size;
    int elem_bytes;
    int num_params;
    int num_groups;
    int kind;                /* ss_layout */
    int has_device_metadata; /* 0 for SS_PLAN_HOST_ONLY plans */
} ss_plan_info;

/* AdamW hyper-parameters for one step (decoupled weight decay), step t >= 1. */
typedef struct {
    double lr;
    double beta1;
    double beta2;
    double eps;
    double weight_decay;
    int64_t step;
} ss_adamw;

/* ---------------------------------------------------------------------- */
/* plans                                                                   */
/* ---------------------------------------------------------------------- */

/* Build a plan ("FSDP1 vs FSDP2", section 03: padding and chunk rules; the
 * flat metadata of numels-with-padding and shapes that split the flat view
 * back into parameters).  Unless SS_PLAN_HOST_ONLY is set, the segment tables
 * are copied to the current device before the call returns.  *out receives
 * the plan; release it with fsdp_plan_destroy.  Errors: SS_EINVAL (sizes,
 * kind, world size, dtype, group counts), SS_EOVERFLOW (a size beyond int64),
 * SS_ENOMEM, SS_ECUDA. */
int fsdp_plan_create(const ss_plan_desc* desc, ss_plan** out);

/* One-group shorthand for fsdp_plan_create (device metadata included). */
int fsdp_plan_layout(ss_layout kind, int world_size, int elem_bytes, int num_params,
                     const int64_t* dim0, const int64_t* inner, ss_plan** out);

/* Geometry of a plan. */
int fsdp_plan_info(const ss_plan* plan, ss_plan_info* out);

/* Where parameter `param` lives in every packed buffer.  FLAT layouts: the
 * element index of its first element (its rank-r elements follow from
 * index / c).  PER_PARAM_DIM0: the element index of its chunk inside rank 0's
 * shard of its group; rank r's chunk is at that index + r*S_g.  chunk_rows_out
 * (nullable) receives c_i for PER_PARAM_DIM0 and 0 for the FLAT layouts. */
int fsdp_plan_param_offset(const ss_plan* plan, int param, int64_t* offset_out,
                           int64_t* chunk_rows_out);

/* Group geometry: base index, elements per rank (S_g or c_g), first parameter
 * and parameter count.  Any output pointer may be NULL. */
int fsdp_plan_group(const ss_plan* plan, int group, int64_t* base_out, int64_t* shard_numel_out,
                    int* first_param_out, int* num_params_out);

/* Self-check of a plan's host tables: every data run lies inside its
 * parameter and its group, the runs cover each parameter element exactly once,
 * data and pad runs tile every packed buffer [0, total_numel) with no gap or
 * overlap, and the tile tables split every run exactly.  The kernels index
 * device memory only through these tables, so a plan that passes keeps every
 * access in bounds.  SS_OK or SS_EINVAL. */
int fsdp_plan_validate(const ss_plan* plan);

/* Free a plan and its device metadata (NULL is a no-op).  The caller makes
 * sure no launch that uses the plan is still pending. */
void fsdp_plan_destroy(ss_plan* plan);

/* ---------------------------------------------------------------------- */
/* step                                                                    */
/* ---------------------------------------------------------------------- */

/*
 * Pack per-parameter tensors into the plan's sharded layout, zero-filling
 * every pad element ("FSDP1 vs FSDP2", section 03: FlatParameter
 * construction; FSDP2's copy-in of a group's shards into one collective
 * buffer).  Used for parameters at initialisation and, per step, for each
 * rank's gradients (the reduce-scatter input).
 *   params  HOST array [num_params] of device pointers; params[i] is the
 *           contiguous tensor of parameter i (numel dim0*inner, the plan's
 *           dtype, aligned to its element size).  Entries of parameters
 *           outside `group` are not read.
 *   packed  device buffer of total_numel elements, 16-byte aligned.  Only the
 *           selected group's range is written.
 *   group   -1 = every group, else one group index.
 * Errors: SS_EINVAL, SS_EALIGN, SS_ENODEVICE, SS_ECUDA.
 */
int fsdp_pack(const ss_plan* plan, const void* const* params, void* packed, int group,
              ss_stream_t stream);

/*
 * Optimizer-state initialisation on every rank's shard: master = the shard
 * widened to fp32, exp_avg = exp_avg_sq = 0 ("Scaling data parallel",
 * section 1: bf16 parameters with an fp32 master copy and fp32 Adam
 * moments).  param_shards: total_numel elements of the plan dtype; master,
 * exp_avg, exp_avg_sq: total_numel floats.  All 16-byte aligned.
 */
int fsdp_init_master(const ss_plan* plan, const void* param_shards, float* master,
                     float* exp_avg, float* exp_avg_sq, int group, ss_stream_t stream);

/*
 * Reduce-scatter of N virtual ranks' gradients fused with AdamW on each
 * rank's shard ("Scaling data parallel", sections 2.1 and 9.1-9.3: the
 * reduce-scatter leaves rank s the sum over ranks of shard s, divided by N
 * for the mean; each rank updates the fp32 master weights and Adam moments
 * of its own 1/N and casts them to bf16; "FSDP1 vs FSDP2", mixed precision:
 * the reduction runs in the reduce dtype, the cast to the parameter dtype
 * happens at the all-gather boundary).
 *
 * For every element f of the selected range (all ranks' shards):
 *   g = (G_0[f] + G_1[f] + ... + G_{N-1}[f]) / N
 * summed in fp32 in rank order starting from G_0, one IEEE fp32 division;
 * then decoupled AdamW (step t = hp->step >= 1):
 *   theta *= 1 - lr*wd;  m = b1*m + (1-b1)*g;  v = b2*v + (1-b2)*g*g;
 *   theta -= (lr / (1-b1^t)) * m / (sqrt(v) / sqrt(1-b2^t) + eps);
 *   param_shards[f] = round-to-nearest-even bf16(theta)   (fp32 plans: theta)
 * in fp32 arithmetic.  Pads hold zero gradients and zero state, and stay zero.
 *
 *   rank_grads        HOST array [N] of device pointers; rank_grads[r] is rank
 *                     r's packed gradient buffer (total_numel elements of the
 *                     plan dtype, as fsdp_pack writes it).
 *   master, exp_avg, exp_avg_sq   total_numel floats, updated in place.
 *                     master may be NULL: the recipe without fp32 master
 *                     weights ("FSDP1 vs FSDP2" ledger: bf16 parameters and
 *                     gradients plus 8 B of Adam moments per parameter).
 *                     theta is then the parameter shard itself, widened to
 *                     fp32, updated, and rounded back in place (2N + 20 bytes
 *                     per element instead of 2N + 26).
 *   param_shards      total_numel elements of the plan dtype, written.
 *   hp                AdamW hyper-parameters; NULL = reduce-scatter only
 *                     (state and shards untouched; reduced_grad_out required).
 *   reduced_grad_out  nullable: total_numel floats receiving g.
 *   group             -1 = every group, else one group index.
 * All device buffers 16-byte aligned and indexed by the same element index.
 * Errors: SS_EINVAL, SS_EALIGN, SS_ENODEVICE, SS_ECUDA.
 */
int fsdp_reduce_scatter_adamw(const ss_plan* plan, const void* const* rank_grads, float* master,
                              float* exp_avg, float* exp_avg_sq, void* param_shards,
                              const ss_adamw* hp, float* reduced_grad_out, int group,
                              ss_stream_t stream);

/*
 * Reduce-scatter with gradient accumulation over num_micro micro-batches per
 * optimizer step ("Scaling data parallel", section 5: accumulate gradients
 * across micro-batches and synchronise once, using their mean; section 9.2:
 * with fp32 accumulation each rank keeps an fp32 gradient for its own shard
 * and adds every reduce-scatter result into it).  With RS_j the reduce-scatter
 * of micro-batch j (as fsdp_reduce_scatter_adamw computes it):
 *   micro_step 0:                 accum = RS_0
 *   0 < micro_step < num_micro-1: accum = accum + RS_j       (fp32)
 *   micro_step = num_micro-1:     g = (accum + RS_j) / num_micro, then AdamW
 *                                 exactly as fsdp_reduce_scatter_adamw
 *                                 (reduced_grad_out, if given, receives g)
 * num_micro = 1 is fsdp_reduce_scatter_adamw.  accum: total_numel floats
 * (16-byte aligned), left holding acc_{k-1} after the last micro-batch.
 * master may be NULL (no-master recipe).  bf16 plans only.
 * Errors: SS_EINVAL, SS_EALIGN, SS_ENODEVICE, SS_ECUDA.
 */
int fsdp_reduce_scatter_accumulate(const ss_plan* plan, const void* const* rank_grads,
                                   float* accum, int micro_step, int num_micro, float* master,
                                   float* exp_avg, float* exp_avg_sq, void* param_shards,
                                   const ss_adamw* hp, float* reduced_grad_out, int group,
                                   ss_stream_t stream);

/*
 * All-gather of the N rank shards followed by unpacking into full
 * per-parameter tensors, pads dropped ("FSDP1 vs FSDP2", section 03 figure:
 * the flat metadata splits the gathered flat view back into parameters;
 * FSDP2 gathers a group's shards in one collective and copies each parameter
 * out).  The all-gather delivers the full parameters to every rank; n_out
 * replicas are written (1 = the copy one rank sees, N = every rank's).
 *   param_shards  total_numel elements (16-byte aligned), rank-major.
 *   params_out    HOST array [n_out * num_params] of device pointers; replica
 *                 j of parameter i is params_out[j*num_params + i] (numel
 *                 dim0*inner, aligned to the element size).
 *   n_out         1..SS_MAX_REPLICAS.
 *   group         -1 = every group, else one group index.
 * Errors: SS_EINVAL, SS_EALIGN, SS_ENODEVICE, SS_ECUDA.
 */
int fsdp_all_gather_unpack(const ss_plan* plan, const void* param_shards,
                           void* const* params_out, int n_out, int group, ss_stream_t stream);

/*
 * The whole sharded step in one pass over the parameters: (copy-in) +
 * reduce-scatter + AdamW + (all-gather + unpack).  Same arithmetic as
 * fsdp_reduce_scatter_adamw followed by fsdp_all_gather_unpack, with
 * bit-identical results, but the kernel knows each element's place inside its
 * parameter (the plan's runs of one parameter inside one rank's shard), so in
 * one pass it can
 *   - read rank r's gradient either from its packed buffer (rank_grads[r],
 *     as fsdp_pack writes it) or straight from rank r's per-parameter
 *     gradient tensors (rank_param_grads[r*num_params + i]), fusing away the
 *     copy-in that FSDP does before its reduce-scatter ("FSDP1 vs FSDP2",
 *     section 04: a group's gradients are concatenated into one
 *     reduce-scatter buffer);
 *   - write each new bf16 parameter value both to its shard and to the n_out
 *     per-parameter outputs (the all-gather + unpack, no second pass over the
 *     shards).
 * Pad elements are not read or written (they stay as fsdp_pack /
 * fsdp_init_master left them: zero).  bf16 plans only.
 * Per-parameter gradients and outputs need only 2-byte alignment: a run at any
 * offset still moves in 16-byte vectors, one side aligned and the other
 * realigned in registers.  With n_out = N the call is the ZeRO-1/2 step
 * ("Scaling data parallel", sections 9.1-9.2): each rank updates its own 1/N
 * and the updated parameters reach every rank.
 */
typedef struct {
    const void* const* rank_grads;        /* HOST [N] packed buffers (16-byte aligned), or NULL */
    const void* const* rank_param_grads;  /* HOST [N * num_params] per-parameter gradients, or NULL;
                                             exactly one of the two is non-NULL */
    float* master;                        /* total_numel floats, updated in place */
    float* exp_avg;
    float* exp_avg_sq;
    void* param_shards;                   /* total_numel bf16, written */
    const ss_adamw* hp;                   /* required */
    float* reduced_grad_out;              /* nullable: total_numel floats (pads not written) */
    void* const* params_out;              /* HOST [n_out * num_params] outputs, or NULL if n_out == 0 */
    int n_out;                            /* 0..SS_MAX_REPLICAS; 0 = no all-gather */
} ss_step;

/* Per launch the pointer table holds (N if rank_param_grads else 0) + n_out
 * entries per parameter within 2048 slots; more parameters are split into
 * launches over consecutive parameters.  Every form runs in one pass and
 * allocates nothing.  Errors: SS_EINVAL (including both or neither gradient
 * source, fp32 plans, (N + n_out) > 2048), SS_EALIGN, SS_ENODEVICE,
 * SS_ECUDA. */
int fsdp_sharded_step(const ss_plan* plan, const ss_step* step, int group, ss_stream_t stream);

/*
 * DDP bucketed gradient average ("Scaling data parallel", sections 3-4:
 * gradients become final last layer first, so tensors are taken in reverse
 * registration order; each joins the open bucket, and a bucket that holds at
 * least bucket_cap_bytes is full and goes out as one all-reduce, the mean
 * over ranks).  For every element of every tensor:
 *   avg_out[t][k] = bf16_rne((g_0 + g_1 + ... + g_{N-1}) / N)
 * summed in fp32 in rank order.  One kernel launch per bucket, in bucket
 * order, so the per-collective fixed cost the pages describe is visible.
 *   world_size    N, 1..SS_MAX_WORLD.
 *   numels        HOST array [num_tensors], each >= 0.
 *   rank_grads    HOST array [N * num_tensors] of device pointers; rank r's
 *                 gradient of tensor t is rank_grads[r*num_tensors + t]
 *                 (bf16, 2-byte aligned).
 *   bucket_cap_bytes  > 0.
 *   avg_out       HOST array [num_tensors] of device pointers (bf16 outputs).
 *   num_buckets_out   nullable: receives the bucket count.
 * The call stages a per-call table of pointers and sizes in device memory
 * obtained with cudaMallocAsync on `stream` and released with cudaFreeAsync
 * after the launches.  The table is copied there from host memory that lives
 * only for the call, so a stream that is being captured into a CUDA graph is
 * refused with SS_EINVAL before anything is queued.
 * Errors: SS_EINVAL, SS_EALIGN, SS_ENOMEM, SS_ECUDA.
 */
int ddp_bucket_pack_average(int world_size, int num_tensors, const int64_t* numels,
                            const void* const* rank_grads, size_t bucket_cap_bytes,
                            void* const* avg_out, int* num_buckets_out, ss_stream_t stream);

/*
 * Allocation-free variant of ddp_bucket_pack_average.  No counterpart on the
 * pages: it exists for callers that cannot call cudaMalloc or
 * cudaMallocAsync -- a host framework that owns every byte of device memory
 * through its own allocator and forbids allocations behind its back, a
 * latency-critical loop that must not risk an allocation that grows a memory
 * pool or synchronises, or a process running so close to its device-memory
 * limit that an allocation could fail in the middle of a step.
 *
 * Same arguments, arithmetic, bucket order and launches as
 * ddp_bucket_pack_average; only the per-call table of pointers and sizes
 * lives in a fixed array inside the library (a static __device__ array of
 * SS_DDP_NOALLOC_TABLE_BYTES that every GPU loading the library holds until
 * the process exits) instead of a cudaMallocAsync allocation.  The table
 * takes 8 * (num_tensors + 1) + 8 * num_tensors * (world_size + 1) bytes; a
 * call that needs more returns SS_ESCRATCH before doing anything.
 *
 * The call allocates no device memory and calls no allocating library
 * routine.  The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and keeps it together with
 * the id of the current CUDA context; a call under another context (after
 * cudaDeviceReset, say) looks it up again.  As for ddp_bucket_pack_average,
 * the table is copied from host memory that lives only for the call, so a
 * stream that is being captured is refused with SS_EINVAL.  Every call
 * overwrites the whole table it uses, so nothing has to be cleared between
 * calls, and calls queued one after another on one stream are ordered by it.
 * All calls share the one array, though: calls whose work can overlap on the
 * GPU (different streams without ordering between them, or several host
 * threads) race on it and must be serialised by the caller.
 */
#define SS_DDP_NOALLOC_TABLE_BYTES (256u * 1024u)
int ddp_bucket_pack_average_noalloc(int world_size, int num_tensors, const int64_t* numels,
                                    const void* const* rank_grads, size_t bucket_cap_bytes,
                                    void* const* avg_out, int* num_buckets_out,
                                    ss_stream_t stream);

/* Bucket assignment only (host, no device work): bucket_of[t] receives
 * tensor t's bucket, numbered in launch order.  Returns the bucket count, or
 * a negative SS_E* status. */
int ddp_bucket_assign(int num_tensors, const int64_t* numels, int elem_bytes,
                      size_t bucket_cap_bytes, int* bucket_of);

/* ---------------------------------------------------------------------- */
/* the loss at the head of the model                                       */
/* ---------------------------------------------------------------------- */

enum { SS_LOSS_MEAN = 0, SS_LOSS_SUM = 1 };

/* ss_linear_ce_workspace flags. */
#define SS_CE_GRADIENT 1u     /* the call writes d_hidden or d_weight */
#define SS_CE_STAGE_WEIGHT 2u /* weight rows not 16-byte aligned (assumed when hidden_size % 8 != 0) */

/*
 * Softmax cross entropy of a linear head, and its gradients, with no logits
 * kept.  With l_tv = <hidden_t, weight_v>, over the tokens t whose target y_t
 * is not ignore_index:
 *   loss_t = log(sum_v exp(l_tv)) - l_t,y_t
 *   loss   = their sum, or their mean (0 when no token counts)
 *   d_hidden, d_weight = grad_scale * the gradient of loss
 * Ignored tokens have a token loss and a d_hidden row of 0, whatever their
 * hidden row holds; a target outside [0, vocab_size) that is not ignore_index
 * makes its token's loss NaN, and with it the loss and the gradients.  So does
 * a logit of NaN or +infinity, of whichever class, and a token whose logits are
 * all -infinity; a target's logit of -infinity is an infinite loss.
 *
 * All matrices are bf16, row-major with a row stride in elements (>= the row's
 * length) and any element alignment; products accumulate and statistics are
 * held in fp32, the logits' exponentials are rounded to bf16 once on their way
 * into the gradients.  Weight rows on 16-byte boundaries (an aligned address
 * and a stride that is a multiple of 8) are read in place, others are copied to
 * the workspace first.  The same inputs give the same bits.
 *
 * Should a wait inside a kernel run out (two seconds; none does but by a fault of
 * the device), the loss is NaN; where it was in the statistics, so are the token
 * losses that count and the gradients, else the gradients are undefined.
 */
typedef struct {
    int64_t num_tokens;   /* T >= 0 */
    int64_t hidden_size;  /* D >= 1 */
    int64_t vocab_size;   /* V >= 1 */
    const void* hidden;   /* [T, D] */
    int64_t hidden_stride;
    const void* weight;   /* [V, D] */
    int64_t weight_stride;
    const int64_t* targets; /* device [T] */
    int64_t ignore_index;
    int reduction;          /* SS_LOSS_MEAN or SS_LOSS_SUM */
    double grad_scale;      /* finite in fp32: the gradient of the objective by the loss */
    float* loss_out;        /* device, 1 float */
    float* token_loss_out;  /* nullable: device [T] */
    void* d_hidden;         /* nullable: [T, D] */
    int64_t d_hidden_stride;
    void* d_weight;         /* nullable: [V, D] */
    int64_t d_weight_stride;
    void* workspace;        /* 256-byte aligned; no contents expected or kept */
    size_t workspace_bytes;
} ss_linear_ce;

/* Bytes of workspace ss_linear_cross_entropy takes for these sizes on the
 * current device. */
int ss_linear_ce_workspace(int64_t num_tokens, int64_t hidden_size, int64_t vocab_size, unsigned flags,
                           size_t* bytes_out);

/* Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW (sizes above 2^28, or strides
 * beyond 64-bit offsets), SS_ECUDA. */
int ss_linear_cross_entropy(const ss_linear_ce* args, ss_stream_t stream);

/* ---------------------------------------------------------------------- */
/* the residual stream between two layers                                  */
/* ---------------------------------------------------------------------- */

/*
 * Dropout.  Of element (r, c) of a [rows, cols] matrix the 16 bits
 *   u = bits 16 (c % 8) .. 16 (c % 8) + 15 of the 128 bits (lowest first) of
 *       Philox4x32-10 with key {seed} and counter {c / 8, r, offset}
 * decide: out = x / (1 - d) where u >= 65536 d, else 0 (whatever x holds), with
 * d = p rounded to a multiple of 2^-16.  No mask is stored: the backward pass is
 * the same call on the gradient.
 *   elem_bytes  2 (bf16) or 4 (fp32): of x and out, row-major with a row stride
 *               in elements (>= cols) and any element alignment.
 *   p           in [0, 1), and not so near 1 that d is 1.
 *   rng         device, {seed, offset}, 64 bits each: read when the call runs, so
 *               that a captured call draws a new mask once they are changed.
 *   out         may be x (with its stride); it overlaps no input otherwise.
 * Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW (2^31 rows, above 2^33 columns,
 * strides beyond 64-bit offsets), SS_ECUDA.
 */
int ss_dropout(int64_t rows, int64_t cols, int elem_bytes, const void* x, int64_t x_stride, void* out,
               int64_t out_stride, double p, const int64_t* rng, ss_stream_t stream);

/*
 * What happens to the residual stream between two layers:
 *   h    = dropout(x) + residual, rounded to the type
 *   rstd = 1 / sqrt(mean over the row of h^2 + eps)
 *   out  = h * rstd * weight
 * without the dropout where its probability is 0 and without the residual where
 * it is NULL; the dropout is ss_dropout's of a [rows, cols] matrix.  Sums and
 * statistics are fp32: a row whose sum of squares passes that (the root of the sum is
 * 1.8e19 or more) is 0, and rstd too; one of zeros is NaN with eps 0.  out is rounded
 * once.  A row that holds a NaN is NaN; beside an infinity, which is NaN itself,
 * the row is 0.  The order of a row's sum, and so the last bits, depends on the
 * sizes, the type, whether mx_data is given, whether every address and row stride is
 * a multiple of 16 bytes, and the device; with these alike, the same inputs give the
 * same bits.
 *
 * All matrices are of the type elem_bytes says (2: bf16, 4: fp32), row-major with
 * a row stride in elements and any element alignment.  sum_out may be x or the
 * residual, out may be x (each with its stride); outputs overlap no input and no
 * other output otherwise.
 */
typedef struct {
    int64_t rows; /* >= 0 */
    int64_t cols; /* 1..32768 */
    int elem_bytes;
    const void* x;
    int64_t x_stride;
    const void* residual; /* nullable */
    int64_t residual_stride;
    const void* weight; /* [cols] */
    double eps;         /* >= 0, finite in fp32 */
    double dropout;     /* probability, as ss_dropout's */
    const int64_t* rng; /* device {seed, offset}; NULL without dropout */
    void* sum_out;      /* nullable: h */
    int64_t sum_stride;
    void* out; /* nullable */
    int64_t out_stride;
    float* rstd_out; /* nullable: device [rows] */
    void* mx_data;   /* nullable: the rows of out as SS_MXFP8, rounded from fp32 */
    void* mx_scales;
} ss_norm;

/* At least one output.  Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW, SS_ECUDA. */
int ss_rms_norm(const ss_norm* args, ss_stream_t stream);

/*
 * Its gradients, of the h and rstd that it left:
 *   n = h * rstd, g = d_out * weight
 *   d_h      = rstd * (g - n * mean over the row of g n) + d_sum: the gradient of
 *              the sum, and so the residual's
 *   d_x      = dropout(d_h), with the mask of the forward pass
 *   d_weight = sum over the rows of d_out * n
 * d_sum (nullable) is the gradient that reaches h from elsewhere.  Sums are fp32,
 * in an order that depends on the sizes, the type, whether every address and row
 * stride is a multiple of 16 bytes, and the device.  d_h may be d_out
 * or d_sum (with its stride); outputs overlap no input and no other output
 * otherwise.
 */
typedef struct {
    int64_t rows;
    int64_t cols; /* 1..32768 */
    int elem_bytes;
    const void* d_out;
    int64_t d_out_stride;
    const void* h;
    int64_t h_stride;
    const void* weight;
    const float* rstd;
    const void* d_sum; /* nullable */
    int64_t d_sum_stride;
    double dropout;
    const int64_t* rng;
    void* d_h; /* nullable */
    int64_t d_h_stride;
    void* d_x; /* nullable */
    int64_t d_x_stride;
    void* d_weight;  /* nullable: [cols] */
    void* workspace; /* with d_weight: 16-byte aligned, no contents expected or kept */
    size_t workspace_bytes;
} ss_norm_grad;

/* Bytes of workspace ss_rms_norm_backward takes on the current device.  Calls that
 * may overlap on the GPU need one each. */
int ss_rms_norm_workspace(int64_t rows, int64_t cols, size_t* bytes_out);

/* At least one output.  Errors: as ss_rms_norm. */
int ss_rms_norm_backward(const ss_norm_grad* args, ss_stream_t stream);

/* ---------------------------------------------------------------------- */
/* matrices in few bits                                                    */
/* ---------------------------------------------------------------------- */

/*
 * Microscaled floats (OCP Microscaling Formats, v1.0): 32 consecutive elements of
 * a row share a power of two; the elements are e2m1 (SS_MXFP4) or e4m3 (SS_MXFP8).
 * The scale of a block is 2^(floor(log2 max|x|) - e), e = 2 or 8 (2^-127 at the
 * least), elements beyond the format's largest (6 or 448) saturate.  A block that
 * holds an infinity or a NaN is NaN throughout.
 *
 * A quantised [rows, cols] matrix is two buffers, 16-byte aligned, of the sizes
 * that ss_mx_bytes tells:
 *   data    row r at r * W * (64 or 128) bytes, W = ceil(cols / 128): its elements,
 *           then zeros to a multiple of 128; of two e2m1 elements in a byte the
 *           first is the low half.
 *   scales  [ceil(rows / 128)][W] tiles of 512 bytes: the scale of row r, block b
 *           (exponent + 127; 255: NaN) at byte 16 (r % 32) + 4 (r % 128 / 32) +
 *           b % 4 of tile [r / 128][b / 4]; 0 for blocks behind the last column.
 *           Those of rows behind the last are not written and do not matter.
 */
enum { SS_MXFP4 = 0, SS_MXFP8 = 1 };

int ss_mx_bytes(int64_t rows, int64_t cols, int format, size_t* data_bytes, size_t* scale_bytes);

/*
 * Quantises a matrix, its transpose, or both from one read.  Elements go to the
 * nearest (ties to even), or, with rng, to one of the two neighbours: up, away from
 * zero, where the part cut off and u / 65536 make 1, u being the 16 bits that
 * ss_dropout takes for the element's place in x (the same for the transpose).  With
 * bf16 inputs the expected value is then the input up to 2^-16 of a step; not so for
 * elements beyond the format's largest (between 6 and 8, or 448 and 512, times the
 * scale), which are cut to it every time, by up to a quarter or an eighth.
 */
typedef struct {
    int64_t rows;
    int64_t cols;
    int elem_bytes; /* of x: 2 (bf16) or 4 (fp32) */
    const void* x;  /* [rows, cols], any element alignment */
    int64_t stride;
    int format;
    void* data; /* nullable with scales */
    void* scales;
    void* t_data; /* nullable with t_scales: the transpose's */
    void* t_scales;
    const int64_t* rng; /* nullable: device {seed, offset} */
} ss_mx_quant;

/* Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW, SS_ECUDA. */
int ss_mx_quantize(const ss_mx_quant* args, ss_stream_t stream);

/* The values that a quantised matrix stands for, rounded to bf16 (elem_bytes 2) or
 * as they are (4).  Errors: as ss_mx_quantize. */
int ss_mx_dequantize(int64_t rows, int64_t cols, int format, const void* data, const void* scales, void* out,
                     int64_t out_stride, int elem_bytes, ss_stream_t stream);

/*
 * out[m, n] = sum over k of A[m, k] B[n, k] of two quantised matrices of one
 * format, [M, K] and [N, K]: a linear layer of a [N, K] weight, and, with transposes
 * from ss_mx_quantize, both its gradients.  Products and sums are the tensor cores'
 * (fp32 accumulators), out is rounded once to bf16 (elem_bytes 2) or fp32 (4).  The
 * same inputs give the same bits.  Should a wait inside the kernel run out (two
 * seconds; none does but by a fault of the device), what it did not reach is NaN.
 */
typedef struct {
    int64_t M;
    int64_t N;
    int64_t K; /* >= 1 */
    int format;
    const void* a_data;
    const void* a_scales;
    const void* b_data;
    const void* b_scales;
    void* out; /* [M, N], any element alignment */
    int64_t out_stride;
    int elem_bytes; /* of out */
} ss_mx_product;

/* Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW (sizes above 2^30), SS_ECUDA. */
int ss_mx_matmul(const ss_mx_product* args, ss_stream_t stream);

/* ---------------------------------------------------------------------- */
/* gradient norm and clipping                                              */
/* ---------------------------------------------------------------------- */

/* Workspace the calls of this section take: device memory, 16-byte aligned,
 * with no contents expected or kept.  Calls that may overlap on the GPU need
 * one each. */
#define SS_NORM_WORKSPACE_BYTES (4u * 1024u * 1024u)

/*
 * Global norm of a list of tensors:
 *   norm_out[0] = n = sqrt(sum over every element of every tensor of x^2)
 *   norm_out[1] = 1
 * Squares and partial sums are fp32, their sum over the CTAs fp64 in a fixed
 * order: the same inputs give the same bits.  NaN and infinities come through
 * (a square passes fp32 from |x| = 1.8e19 on, and vanishes below 2.6e-23); an
 * empty list has norm 0.
 *   numels      HOST array [num_tensors], each >= 0.
 *   elem_bytes  HOST array [num_tensors]: 2 (bf16) or 4 (fp32), in any mixture.
 *   grads       HOST array [num_tensors] of device pointers to contiguous
 *               tensors, aligned to their element size; those of empty tensors
 *               are not looked at.
 *   norm_out    device, 2 floats.
 * Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW, SS_ECUDA.
 */
int ss_grad_norm(int num_tensors, const int64_t* numels, const int* elem_bytes,
                 const void* const* grads, float* norm_out, void* workspace, size_t workspace_bytes,
                 ss_stream_t stream);

/*
 * The same norm, and every tensor scaled by the clipping factor:
 *   norm_out[1] = c = min(1, max_norm / (n + 1e-6))   (NaN where n is)
 *   out[k] = c * grads[k], in fp32, rounded once to the tensor's type
 *   out         HOST array [num_tensors] of device pointers, or NULL for in
 *               place.  Each is its own input's address or overlaps no input
 *               and no other output; any element alignment.
 *   max_norm    >= 0; +infinity never clips (c is 1 for an infinite norm too).
 * In place, nothing is written when c is 1.
 * Errors: as ss_grad_norm.
 */
int ss_clip_grads(int num_tensors, const int64_t* numels, const int* elem_bytes, void* const* grads,
                  void* const* out, double max_norm, float* norm_out, void* workspace,
                  size_t workspace_bytes, ss_stream_t stream);

/*
 * Reduce-scatter of N virtual ranks' gradients with the sum of the result's
 * squares: what a sharded step does per group while gradients arrive, before
 * the norm over all groups is known.
 *   reduced_grad[f] = g = (G_0[f] + ... + G_{N-1}[f]) / N, bit for bit the g of
 *                     fsdp_reduce_scatter_adamw
 *   *sq_out         = sum of g^2 over the selected range (pads hold zero
 *                     gradients and add nothing); 0 for an empty one
 *   rank_grads    HOST array [N] of packed gradient buffers of the plan dtype,
 *                 16-byte aligned.
 *   reduced_grad  total_numel floats, 16-byte aligned.
 *   sq_out        device, 1 double.
 *   group         -1 = every group, else one group index.
 * Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW, SS_ENODEVICE, SS_ECUDA.
 */
int fsdp_reduce_scatter_norm(const ss_plan* plan, const void* const* rank_grads, float* reduced_grad,
                             double* sq_out, void* workspace, size_t workspace_bytes, int group,
                             ss_stream_t stream);

/*
 * AdamW on the clipped reduced gradient of the selected range:
 *   n = sqrt(sum of sq_sums), c = min(1, max_norm / (n + 1e-6)); norm_out = {n, c}
 *   g = c * reduced_grad[f], then AdamW exactly as fsdp_reduce_scatter_adamw
 * With c = 1 the state and shards are bit for bit what fsdp_reduce_scatter_adamw
 * gives.
 *   sq_sums       device, num_sums doubles, summed in a fixed order: the sq_out of
 *                 every group (and of other plans whose gradients the norm
 *                 spans).
 *   max_norm      >= 0; +infinity never clips (c is 1 for an infinite norm too).
 *   master        nullable: the recipe without fp32 master weights.
 *   norm_out      device, 2 floats.
 * The other arguments are fsdp_reduce_scatter_adamw's; bf16 and fp32 plans.
 * Errors: SS_EINVAL, SS_EALIGN, SS_EOVERFLOW, SS_ENODEVICE, SS_ECUDA.
 */
int fsdp_clip_adamw(const ss_plan* plan, const float* reduced_grad, const double* sq_sums, int num_sums,
                    double max_norm, float* master, float* exp_avg, float* exp_avg_sq,
                    void* param_shards, const ss_adamw* hp, float* norm_out, int group,
                    ss_stream_t stream);

/* ---------------------------------------------------------------------- */
/* diagnostics                                                             */
/* ---------------------------------------------------------------------- */

/* Static description of a status code. */
const char* ss_strerror(int status);

/* cudaError_t recorded by the last SS_ECUDA returned on this thread (0 if none). */
int ss_last_cuda_error(void);

/* Library version, e.g. "0.1.0". */
const char* ss_version(void);

/* Number of kernels this library has launched in this process (all devices,
 * all threads), for accounting launches inside a timed region. */
uint64_t ss_launch_count(void);

/* For testing how a kernel that gives up is reported: this process's next
 * ss_linear_cross_entropy call gets a wait that nothing ends, and that runs out,
 * in its tensor-core launch number `launch` -- 0 forms the statistics, the ones
 * from 1 on the gradients -- where the call makes that launch.  -1: none.
 * Everything else of the launch runs as always.  Errors: SS_EINVAL. */
int ss_linear_ce_expire_wait(int launch);

/* The same for this process's next ss_mx_matmul call that launches (on 1; 0: none):
 * the first CTA, or pair of CTAs, waits before its products for what never comes, and
 * the tiles of out that are its own are NaN.  Errors: SS_EINVAL. */
int ss_mx_expire_wait(int on);

#ifdef __cplusplus
}
#endif

#endif /* SHARDSTATE_H */
