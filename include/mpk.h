/*
 * mpk.h -- C ABI of the GB300 (sm_103a) mega-kernel decode runtime.
 *
 * One LLM decode step is compiled into a task/event graph (tGraph) and run
 * inside one persistent kernel: "MPK: A Compiler and Runtime for
 * Mega-Kernelizing Tensor Programs" (§2 Q2, §4, Table 1).  Two calls carry
 * the method: mpk_build_tgraph (model shape + tile sizes -> tGraph) and
 * mpk_decode_step (graph + tokens + paged KV cache + stream -> one step).
 *
 * Conventions for every call:
 *   - All tensors are row-major.  bf16 tensors are IEEE bfloat16 bit
 *     patterns (uint16).  Pointers named d_* and every pointer inside
 *     mpk_weights / mpk_kv_cache are CUDA device pointers on the device that
 *     is current when mpk_bind_weights is called; all other pointers are host
 *     pointers.
 *   - Ownership: the caller owns weights, KV pools, page tables, seq_lens,
 *     tokens, logits and next-token buffers, and keeps them alive while the
 *     graph uses them (pointers are borrowed, never copied or freed).  The
 *     library owns the graph, its device encoding (descriptors, queues,
 *     counters) and the activation workspace, all released by
 *     mpk_destroy_tgraph.
 *   - Errors: host-detectable errors are returned synchronously and leave
 *     the graph unchanged.  Errors detected inside the kernel (a bounded wait
 *     that ran out, an unmapped KV page, a full queue) are latched in a
 *     device status word that mpk_get_status reads; the kernel then exits
 *     cleanly and the graph needs mpk_reset before the next step.
 *   - Threading: no global state.  One graph is used by one host thread and
 *     one stream at a time; distinct graphs are independent.
 */
#ifndef MPK_H_
#define MPK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MPK_OK = 0,
  MPK_ERR_INVALID_ARG = 1,     /* a null pointer, a non-positive size, ... */
  MPK_ERR_UNSUPPORTED = 2,     /* a shape the task bodies do not handle    */
  MPK_ERR_CUDA = 3,            /* a CUDA runtime/driver call failed         */
  MPK_ERR_OOM = 4,             /* device or host allocation failed          */
  MPK_ERR_NOT_CORESIDENT = 5,  /* workers + schedulers exceed the SMs, or
                                  the persistent grid cannot be co-resident */
  MPK_ERR_TIMEOUT = 6,         /* a bounded device wait ran out             */
  MPK_ERR_KV_PAGE = 7,         /* page_table holds -1 where a token lives   */
  MPK_ERR_QUEUE_OVERFLOW = 8,  /* a device queue could not take an entry    */
  MPK_ERR_GRAPH_INVALID = 9,   /* the built graph failed its invariants     */
  MPK_ERR_NOT_BOUND = 10       /* decode before mpk_bind_weights            */
} mpk_status;

/* Model shape.  Decoder mode: n_layers >= 1, chain_ffn == 0.  Chained-linear
 * mode: n_layers == 0 and chain_ffn > 0; the step is then
 * x = embed[token]; n = RMSNorm(x, final_norm); y = silu(n W1^T);
 * z = y W2^T; logits = z lm_head^T (no KV cache, no attention). */
typedef struct {
  int n_layers;
  int hidden;
  int n_q_heads;
  int n_kv_heads;
  int head_dim;          /* even, <= 128                                   */
  int ffn;               /* SwiGLU intermediate size                        */
  int vocab;
  float rms_eps;
  float rope_theta;
  int qk_norm;           /* 1: per-head RMSNorm of q and k before RoPE      */
  int chain_ffn;         /* > 0 selects the chained-linear mode             */
  int page_size;         /* KV tokens per page                              */
  int max_pages_per_seq; /* columns of the page table                       */
} mpk_model_shape;

/* Tile sizes and runtime geometry; 0 selects the default. */
typedef struct {
  int num_workers;        /* W worker SMs.  0: the SM count of the current
                             device minus num_sched_sms (needs a GPU)       */
  int gemv_rows_per_task; /* MatMul output rows per task at batch < 8 (a
                             multiple of 8).  0: T = W * ceil(ceil(N/cap)/W)
                             tiles (at most ceil(N/8)) of multiples of 8
                             rows (single rows at batch 1).  cap at batch 1:
                             2560 / p rows, p = the partial sums a row's dot
                             product is split into (1 when a 32 KB page
                             holds r = max(1, 16384 / K) >= 8 rows, else
                             8 / r); 64 at batch 2..7; a gate/up row counts
                             twice; rounded down to a multiple of 8        */
  int mma_rows_per_task;  /* the same for batch >= 8, where MatMul tiles run
                             on tensor cores; 0: as above with cap = 128    */
  int attn_chunks;        /* split-KV chunks per (sequence, KV head).  0:
                             max(1, min(ceil(max_ctx/128),
                             ceil(4W/(batch*n_kv_heads))))                  */
  int num_sched_sms;      /* SMs running scheduler warps.  0: 4 (Table 1)
                             when the graph has JIT tasks, none when every
                             task is AOT (no dispatch: all SMs are workers) */
  int sched_warps_per_sm; /* 0: 4 (Table 1)                                 */
  int smem_pages;         /* weight pages per worker (batch 1: 32 KB of
                             whole rows; batch > 1: 8 rows x 2048 columns,
                             32 KB + row skew). 0: as many as fit, <= 6    */
  int coarse_events;      /* 1: every task of an operator waits for every
                             task of the operators it reads (the
                             operator-level graph of Figure 4c, an
                             ablation); 0: region-overlap events           */
} mpk_tile_sizes;

/* Task kinds (one per operator of the decode step). */
enum {
  MPK_TASK_EMPTY = 0,     /* normalisation glue: waits, then triggers      */
  MPK_TASK_QKV = 1,       /* MatMul tile of W_qkv; prologue: residual add
                             (layer 0: embedding gather) + RMSNorm          */
  MPK_TASK_ATTN = 2,      /* one KV chunk of one (sequence, KV head): q/k
                             RMSNorm (optional) + RoPE + KV append, paged
                             attention over the chunk, and the log-sum-exp
                             merge of all chunks by the last to finish     */
  MPK_TASK_O = 3,         /* MatMul tile of W_o                             */
  MPK_TASK_GATEUP = 4,    /* MatMul tile of W_gate and W_up; prologue:
                             residual add + RMSNorm; epilogue: SwiGLU       */
  MPK_TASK_DOWN = 5,      /* MatMul tile of W_down                          */
  MPK_TASK_LM_HEAD = 6,   /* MatMul tile of lm_head (prologue: final norm),
                             fp32 logits + tile argmax                      */
  MPK_TASK_ARGMAX = 7,    /* argmax over tile maxima; seq_lens += 1         */
  MPK_TASK_CHAIN_UP = 8,  /* MatMul tile of W1 (prologue: RMSNorm) + SiLU   */
  MPK_TASK_CHAIN_DOWN = 9,
  MPK_TASK_NKINDS = 10
};

/* Launch classes (hybrid JIT/AOT, MPK summary §2 Q2 and "Design space"). */
enum {
  MPK_LAUNCH_AOT = 0,     /* statically placed on one worker's queue        */
  MPK_LAUNCH_JIT = 1,     /* placed by a scheduler warp when its event fires*/
  MPK_LAUNCH_INLINE = 2   /* empty task, run by whoever fires its event     */
};

/* Execution modes of mpk_decode_step. */
enum {
  MPK_MODE_MEGAKERNEL = 0,  /* one persistent launch per step (default)     */
  MPK_MODE_KPO = 1,         /* one launch per operator, same task bodies    */
  MPK_MODE_KPO_GRAPH = 2    /* the KPO launches replayed from a CUDA Graph  */
};

/* Per-layer weight tensors, in the order of mpk_weights.layers. */
enum {
  MPK_W_LN1 = 0,     /* bf16 [hidden]                                       */
  MPK_W_QKV = 1,     /* bf16 [(Hq + 2 Hkv) d][hidden]: q heads, k heads, v  */
  MPK_W_QNORM = 2,   /* bf16 [d] (qk_norm only, else ignored)               */
  MPK_W_KNORM = 3,   /* bf16 [d] (qk_norm only, else ignored)               */
  MPK_W_O = 4,       /* bf16 [hidden][Hq d]                                 */
  MPK_W_LN2 = 5,     /* bf16 [hidden]                                       */
  MPK_W_GATEUP = 6,  /* bf16 [2 ffn][hidden]: rows [0,ffn) gate, then up    */
  MPK_W_DOWN = 7,    /* bf16 [hidden][ffn]                                  */
  MPK_LAYER_NTENSORS = 8
};

typedef struct mpk_graph mpk_graph; /* opaque, library-owned */

/* Device weight pointers (borrowed).  Every bf16 tensor must be 16-byte
 * aligned.  `layers` is a HOST array of n_layers * MPK_LAYER_NTENSORS device
 * pointers, read during the call only. */
typedef struct {
  const void* embed;           /* bf16 [vocab][hidden]                       */
  const void* final_norm;      /* bf16 [hidden]                              */
  const void* lm_head;         /* bf16 [vocab][hidden]                       */
  const void* const* layers;   /* decoder mode                               */
  const void* chain_w1;        /* chained mode: bf16 [chain_ffn][hidden]     */
  const void* chain_w2;        /* chained mode: bf16 [hidden][chain_ffn]     */
} mpk_weights;

/* Paged KV cache (caller-owned device memory).  Token t of sequence b lives
 * in page page_table[b][t / page_size] at slot t % page_size. */
typedef struct {
  void* k_pool;                /* bf16 [n_layers][num_pages][Hkv][page_size][d] */
  void* v_pool;                /* same layout                                */
  const int32_t* page_table;   /* int32 [batch][max_pages_per_seq], -1 = none */
  int32_t* seq_lens;           /* int32 [batch]: tokens already cached       */
  int num_pages;
} mpk_kv_cache;

/* Host arrays describing a built graph, owned by the graph (valid until
 * mpk_destroy_tgraph).  Tasks and events are in linearised order. */
typedef struct {
  int n_tasks, n_events, n_ops, n_empty, n_workers, attn_chunks;
  const int32_t* task_kind;    /* MPK_TASK_*                                 */
  const int32_t* task_op;      /* operator index, -1 for empty tasks         */
  const int32_t* task_layer;   /* layer (n_layers for the final operators)   */
  const int32_t* task_tile;    /* tile index within its operator             */
  const int32_t* task_row0;    /* MatMul: output rows [row0, row1)           */
  const int32_t* task_row1;
  const int32_t* task_b;       /* attention family: sequence, KV head, chunk */
  const int32_t* task_g;
  const int32_t* task_c;
  const int32_t* task_dep;     /* the one event the task waits on            */
  const int32_t* task_trig;    /* the one event the task triggers            */
  const int32_t* task_launch;  /* MPK_LAUNCH_*                               */
  const int32_t* task_worker;  /* AOT worker, -1 otherwise                   */
  const int32_t* task_pre_id;  /* id before linearisation (program order)    */
  const int32_t* event_count;  /* triggers needed to activate the event      */
  const int32_t* event_first;  /* dependent tasks are [first, last]          */
  const int32_t* event_last;
  const int32_t* op_kind;      /* per operator, in program order             */
  const int32_t* op_layer;
  const int32_t* op_n_tasks;
  int64_t n_raw_events;        /* events before fusion                       */
  int64_t n_fused_events;      /* events after fusion, before normalisation  */
  int n_sched_sms;             /* scheduler SMs of the launch (0: all-AOT)   */
  int sched_warps_per_sm;
} mpk_graph_export;

/* Decompose one decode step of `shape` at `batch` sequences into per-tile
 * tasks, derive events from overlapping output/input regions, fuse them
 * (Defs 4.1 and 4.2), normalise (<= 1 dependent and <= 1 triggering event
 * per task) and BFS-linearise (each event's fan-out is [first, last]).
 * MPK summary §2 Q2 and §4 "6 minimum checks".  Host only: touches no GPU
 * unless tiles->num_workers == 0.  On success *out owns a new graph. */
mpk_status mpk_build_tgraph(const mpk_model_shape* shape,
                            const mpk_tile_sizes* tiles, int batch,
                            mpk_graph** out);

/* Copy the graph's device encoding to the current device, allocate the
 * activation workspace and bind the weights (pointers borrowed).  May be
 * called again to rebind other weights of the same shape. */
mpk_status mpk_bind_weights(mpk_graph* g, const mpk_weights* w);

/* Enqueue one decode step on `cuda_stream` (a cudaStream_t, 0 = legacy
 * default stream): d_tokens int32 [batch] in; d_logits fp32 [batch][vocab]
 * and d_next_tokens int32 [batch] (greedy, lowest index on ties) out.  Reads
 * kv->seq_lens[b] as the position of the new token, writes its K/V there,
 * and on success increments seq_lens in the kernel.  Asynchronous: returns
 * after the launch(es) are enqueued.  In megakernel mode this is one
 * cooperative launch of a persistent grid (MPK summary, Figure 1: "a
 * single launch").  d_tokens may alias the previous step's d_next_tokens. */
mpk_status mpk_decode_step(mpk_graph* g, const int32_t* d_tokens,
                           const mpk_kv_cache* kv, float* d_logits,
                           int32_t* d_next_tokens, void* cuda_stream);

/* Several greedy steps in ONE launch (MPK summary, Figure 1: the whole
 * decode loop inside a single launch).  Step i (0 <= i < n_steps) embeds
 * d_tokens for i = 0, else the tokens step i - 1 wrote; it writes its own to
 * d_next_tokens + i * batch (device int32 [n_steps][batch]).  d_logits
 * receives the last step's logits.  kv and seq_lens advance by n_steps.
 * Inside the kernel every worker walks its task queue once per step: the
 * first tasks of step i + 1 wait for step i's end event, while the
 * producers already stream step i + 1's weights during step i's last tasks
 * (cached K/V pages only after that end event).  In the kernel-per-operator
 * modes the steps are enqueued one after another.  Same errors and
 * asynchrony as mpk_decode_step; n_steps < 1 is MPK_ERR_INVALID_ARG. */
mpk_status mpk_decode_steps(mpk_graph* g, const int32_t* d_tokens,
                            const mpk_kv_cache* kv, float* d_logits,
                            int32_t* d_next_tokens, int n_steps,
                            void* cuda_stream);

/* Read the device status word of the last step.  Synchronises the device.
 * MPK_OK, or the first error the kernel latched. */
mpk_status mpk_get_status(mpk_graph* g);

/* Select MPK_MODE_MEGAKERNEL, MPK_MODE_KPO or MPK_MODE_KPO_GRAPH. */
mpk_status mpk_set_mode(mpk_graph* g, int mode);

/* Fill *out with host arrays of the built graph (for parity checks). */
mpk_status mpk_export_tgraph(const mpk_graph* g, mpk_graph_export* out);

/* Clear the device status, abort flag, event counters and queues after an
 * error (synchronises the device).  The KV cache is the caller's to fix. */
mpk_status mpk_reset(mpk_graph* g);

/* Free everything the graph owns.  Null is ignored. */
void mpk_destroy_tgraph(mpk_graph* g);

const char* mpk_status_string(mpk_status s);

/* Test hooks.  mpk_debug_set_wait_timeout_ms bounds every device wait of
 * later steps (default 2000 ms).  mpk_debug_add_event_count adds `delta` to
 * the trigger count of linearised event `event` in the device encoding, so a
 * test can make a wait that never completes and check MPK_ERR_TIMEOUT. */
mpk_status mpk_debug_set_wait_timeout_ms(mpk_graph* g, int ms);
mpk_status mpk_debug_add_event_count(mpk_graph* g, int event, int delta);

/* Tracing (megakernel mode).  mpk_debug_set_trace(g, capacity) allocates
 * room for `capacity` task records (0 disables).  Each executed task adds one
 * record of eight uint64: task id | (worker << 32), then the %globaltimer
 * nanoseconds at which the worker's leader started looking for it, found it
 * ready, had its operands staged (batch-1 MatMul tiles; else 0), had
 * consumed its last weight page (batch-1 MatMul tiles; else 0), finished its
 * body, and finished its trigger; the eighth word is 0.
 * mpk_debug_read_trace copies up to `capacity` records into host_records,
 * stores the count, and clears the trace for the next steps (synchronises
 * the device). */
mpk_status mpk_debug_set_trace(mpk_graph* g, int capacity);
mpk_status mpk_debug_read_trace(mpk_graph* g, uint64_t* host_records,
                                int capacity, int* n_records);

/* Copy the residual stream entering decoder layer `layer` of the last step
 * (0 <= layer <= n_layers; n_layers is the input of the final RMSNorm) into
 * host_out, bf16 [batch][hidden] (synchronises the device).  The first
 * MatMul tile of each layer (and of lm_head) stores it as a by-product of
 * its RMSNorm prologue.  Decoder mode only. */
mpk_status mpk_debug_read_hidden(mpk_graph* g, int layer, uint16_t* host_out);

/* CPU model of the runtime protocol (no GPU needed).  Runs `steps` steps
 * of g's own device encoding with one host thread per worker leader and per
 * scheduler warp: epoch counters, AOT queues in linear order (with the
 * cached fan-outs of the AOT records), JIT dispatch through scheduler and
 * worker rings, and empty tasks run inline by the activating trigger, as
 * the kernel does (MPK summary, §2 Q2 runtime; Figure 8).  Task bodies
 * are replaced by random delays of 0..max_delay_us microseconds (seeded).
 * Reports, in *report: executions, executions that started before some
 * task triggering their event had finished in the same step, duplicate and
 * missing executions per completed step, and whether a step failed to
 * finish within timeout_ms (a deadlock).  Returns MPK_ERR_INVALID_ARG for
 * bad arguments; the verdict is in the report. */
typedef struct {
  int64_t tasks_run;
  int64_t order_violations;
  int64_t duplicate_runs;
  int64_t missing_runs;
  int32_t deadlocked;
  int32_t steps_completed;
  double seconds;
} mpk_sim_report;
mpk_status mpk_debug_simulate(const mpk_graph* g, int steps, uint32_t seed,
                              int max_delay_us, int timeout_ms,
                              mpk_sim_report* report);

/* Allocation-free decode step.  (The paper has no counterpart: this is a
 * convenience for callers of the library.)
 *
 * For callers that cannot call cudaMalloc while they run: a serving process
 * whose device memory is reserved up front by its own caching allocator, a
 * latency-critical loop that may not take the device-wide synchronisation
 * cudaMalloc/cudaFree imply, or a plugin whose host owns every allocation.
 * The call runs the kernel-per-operator form of the step (the same task
 * bodies as mpk_decode_step) and keeps all of its scratch -- task
 * descriptors, the layer pointer table, the RoPE table, the attention merge
 * counters, the activation workspace and the status words -- in one static
 * device array of MPK_NOALLOC_SCRATCH_BYTES that every
 * GPU loading the library holds until the process exits.  It calls no
 * cudaMalloc, cudaFree or other allocating routine.
 *
 * g comes from mpk_build_tgraph (mpk_bind_weights is not needed); w, d_tokens,
 * kv, d_logits and d_next_tokens are as for mpk_bind_weights and
 * mpk_decode_step, on the current device.  d_status (nullable, device
 * uint32) receives the step's mpk_status once the step has run.
 * Returns MPK_ERR_UNSUPPORTED, before touching the device, when the graph
 * needs more scratch than MPK_NOALLOC_SCRATCH_BYTES (8 MiB: e.g. the tiny,
 * ~1B-parameter and chained-linear shapes fit, the 36-layer 8B shape does
 * not).  The first call on a device looks up the array's device address,
 * so make that first call before any stream capture.  All calls share the
 * one array, which keeps the last call's contents: calls that overlap on
 * the GPU (other streams, or other host threads) race and must not be
 * issued.  Asynchronous on cuda_stream. */
#define MPK_NOALLOC_SCRATCH_BYTES (8u << 20)
mpk_status mpk_decode_step_noalloc(const mpk_graph* g, const mpk_weights* w,
                                   const int32_t* d_tokens,
                                   const mpk_kv_cache* kv, float* d_logits,
                                   int32_t* d_next_tokens, uint32_t* d_status,
                                   void* cuda_stream);

/* ---------------------------------------------------------------------
 * Serving operators over the paged KV cache: several new tokens a sequence.
 * (The paper's step takes one token a sequence; these calls are what a
 * server puts around it: prompts, shared prompts, drafted tokens.)
 *
 * Three calls make one step of drafted decoding of a layer and of a batch:
 *   mpk_kv_append         norm and rotate the new tokens' q and k, append k, v
 *   mpk_prefix_attention  the new tokens' attention over the cache
 *   mpk_verify_drafts     accept or refuse the drafts, sample the next token
 * and mpk_verify_step runs a built graph's whole step with them.
 *
 * All of them are asynchronous on `cuda_stream`, allocate nothing and can be
 * captured into a CUDA graph.  Pointers are device pointers of the current
 * device unless said otherwise.  Calls that may run at the same time (other
 * streams, other captured graphs) need workspaces of their own; a workspace
 * needs no initialisation and holds nothing between calls.
 * `d_status` (nullable, uint32) keeps the first error a kernel finds (the
 * kernels only replace MPK_OK; the caller clears it).  After an error the
 * results of the sequences (for a prefix: of the group) concerned are
 * unspecified, those of the others are right, and no memory outside the
 * arguments' is touched. */

/* Heads of one layer and the geometry of its cache (mpk_kv_cache layout).
 * head_dim is 32, 64 or 128; n_q_heads a multiple of n_kv_heads; page_size
 * times max_pages_per_seq at most 2^30; the pools' num_pages x n_kv_heads x
 * page_size rows of a layer fewer than 2^32. */
typedef struct {
  int n_q_heads;
  int n_kv_heads;
  int head_dim;
  int page_size;
  int max_pages_per_seq;
} mpk_attn_shape;

/* The new tokens of a batch, as the rows of token-major tensors.  Sequence b
 * owns rows [q_start[b], q_start[b + 1]), none if the two are equal; with a
 * null q_start it owns [b * tokens_per_seq, (b + 1) * tokens_per_seq).  Row i
 * of sequence b (from 0) stands at position seq_lens[b] + i.  Rows outside
 * every sequence (padding behind the last) are neither read nor written. */
typedef struct {
  int batch;
  int n_tokens;             /* rows of the tensors                          */
  const int32_t* q_start;   /* nullable, int32 [batch + 1], ascending       */
  int tokens_per_seq;
} mpk_token_batch;

/* Rotary positions.  The table is fp32 [n_pos][rotary_dim / 2][2] (cos, sin),
 * row p for position p (mpk_rope_table writes one; mpk_decode_step's own is
 * the one of scaling MPK_ROPE_PLAIN).  The first rotary_dim values of a head
 * are rotated (a multiple of 16, at most head_dim; 0: none), in pairs
 * (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved != 0. */
typedef struct {
  const float* table;
  int n_pos;
  int rotary_dim;
  int interleaved;
} mpk_rope;

/* Scaling of the frequencies f_i = theta^(-2i / rotary_dim) for contexts
 * longer than the trained old_ctx. */
enum {
  MPK_ROPE_PLAIN = 0,   /* f_i                                              */
  MPK_ROPE_LINEAR = 1,  /* f_i / factor                                     */
  MPK_ROPE_BANDS = 2,   /* a mixture of f_i / factor and f_i by the turns
                           t_i = old_ctx f_i / 2 pi a pair makes: all of the
                           first for t_i <= low, of the second for
                           t_i >= high, linear in t_i between               */
  MPK_ROPE_RAMP = 3     /* the same mixture, linear in i between (the whole
                           numbers around) the indices of high and low turns */
};
typedef struct {
  int rotary_dim;
  double theta;
  int scaling;            /* MPK_ROPE_*                                     */
  double factor;          /* > 0; unused by MPK_ROPE_PLAIN                  */
  double low, high;       /* 0 < low < high  (BANDS, RAMP)                  */
  double old_ctx;         /* > 0             (BANDS, RAMP)                  */
  double attn_factor;     /* multiplies every cos and sin; 0 means 1        */
} mpk_rope_scaling;

/* Write rows [first_pos, first_pos + n_pos) of a rotation table to d_table
 * (fp32 [n_pos][rotary_dim / 2][2]).  Angles are formed in 64 bits. */
mpk_status mpk_rope_table(const mpk_rope_scaling* s, int64_t first_pos,
                          int n_pos, float* d_table, void* cuda_stream);

/* New tokens into layer `layer` of the cache.  d_q, d_k, d_v: bf16 rows of
 * heads, [n_tokens][heads * head_dim] with row strides in elements (the
 * parts of a fused projection's rows, or separate tensors).  q and k get a
 * per-head RMSNorm with gains d_q_norm / d_k_norm (bf16 [head_dim], nullable:
 * none; rounded to bf16) and the rotation of *rope (nullable: none), with the
 * arithmetic and roundings of mpk_decode_step; v goes in as it is.  Rotated q
 * goes to d_q_out (its own row stride; it may be d_q itself; null: q is not
 * touched).  seq_lens is read, not advanced.  Pointers 16-byte aligned,
 * strides multiples of 8.
 * Errors in d_status: MPK_ERR_KV_PAGE for a position without a page,
 * MPK_ERR_INVALID_ARG for one past the table; such a token is skipped. */
mpk_status mpk_kv_append(const mpk_attn_shape* shape,
                         const mpk_token_batch* tok, const mpk_kv_cache* kv,
                         int layer, const void* d_q, int64_t q_stride,
                         const void* d_k, int64_t k_stride, const void* d_v,
                         int64_t v_stride, const void* d_q_norm,
                         const void* d_k_norm, float eps,
                         const mpk_rope* rope, void* d_q_out,
                         int64_t q_out_stride, uint32_t* d_status,
                         void* cuda_stream);

/* Groups of consecutive sequences that share their first tokens: group g is
 * sequences [group_start[g], group_start[g + 1]), ascending from 0 to the
 * batch, and positions [0, prefix_len[g]) of all of them hold the same keys
 * and values; these are read through the page table row of the group's
 * FIRST sequence, once for the whole group (the other rows may map the same
 * pages or anything else there).  Every sequence of the group with new tokens
 * must have seq_lens >= prefix_len (else MPK_ERR_INVALID_ARG in d_status).
 * A prefix_len of 0 is no prefix. */
typedef struct {
  int n_groups;                /* 1 .. batch                                */
  const int32_t* group_start;  /* device int32 [n_groups + 1]               */
  const int32_t* prefix_len;   /* device int32 [n_groups]                   */
} mpk_prefix_groups;

/* Bytes of workspace that mpk_prefix_attention needs (0 for arguments that
 * it refuses).  n_groups: 0 without groups. */
size_t mpk_prefix_attention_workspace(const mpk_attn_shape* shape,
                                      const mpk_token_batch* tok,
                                      int n_groups);

/* Attention of the new tokens of layer `layer`, whose keys and values are in
 * the cache already (mpk_kv_append): row at position t sees keys 0..t.
 * d_q bf16 [n_tokens][n_q_heads * head_dim] (row stride in elements), d_out
 * the same (its own stride; not d_q), d_lse (nullable) fp32
 * [n_tokens][n_q_heads]: log of the row's sum of exponentials.  Query head j
 * reads KV head j / (n_q_heads / n_kv_heads).  scale multiplies the scores;
 * 0 selects 1/sqrt(head_dim).  groups may be null.  A row that sees no key
 * gives zeros and -inf.  Values that are not finite at keys a row does not
 * see do not reach it.  Pointers 16-byte aligned (d_lse 4), strides
 * multiples of 8; d_workspace 256-byte aligned.  At most 2^20 sequences. */
mpk_status mpk_prefix_attention(const mpk_attn_shape* shape,
                                const mpk_token_batch* tok,
                                const mpk_prefix_groups* groups,
                                const mpk_kv_cache* kv, int layer,
                                const void* d_q, int64_t q_stride, float scale,
                                void* d_out, int64_t out_stride, float* d_lse,
                                void* d_workspace, size_t workspace_bytes,
                                uint32_t* d_status, void* cuda_stream);

/* Inputs and outputs of mpk_verify_drafts.  Row i of sequence b holds token
 * tokens[row] (i = 0: the last token accepted before, i >= 1: draft i), and
 * logits[row] are the model's after that token, so row i judges draft i + 1
 * and a sequence of n rows has n - 1 drafts (at most 127).  A draft outside
 * [0, vocab) ends its sequence's drafts (as if all before it were all).
 * p = softmax(logits / T).  draft row i says what draft i + 1 was drawn from:
 * probabilities, or (draft_is_logits) logits taken at the same T; null: the
 * drafts were chosen outright, q = 1.  Draft i + 1 is accepted when
 * uniform[row i] * q < p; at the first refusal the next token is
 * argmax_v max(p_v - q_v, 0) / noise[b][v] (p alone where that is nowhere
 * positive; without `draft`, p without the refused token), and with all
 * accepted argmax_v p_v / noise[b][v] of the last row; ties take the lowest
 * index.  Outputs overlap no inputs, but for seq_lens_out.  With uniform in
 * [0, 1) and noise ~ Exp(1), the emitted tokens are
 * distributed as samples of p.  T <= 0 (or NaN) is greedy: a draft is accepted
 * when it is the row's argmax, the next token is the argmax; other T count as
 * the nearest of [1e-30, 1e30].  NaN logits count as
 * -inf, several +inf share the row; a row of nothing but -inf accepts nothing
 * and gives token -1. */
typedef struct {
  int vocab;
  int max_out;               /* columns of out_tokens, >= rows of a sequence */
  const int32_t* tokens;     /* [n_tokens]                                  */
  const float* logits;       /* [n_tokens], row stride logits_stride        */
  int64_t logits_stride;     /* elements                                    */
  const float* draft;        /* nullable [n_tokens], row stride draft_stride */
  int64_t draft_stride;
  int draft_is_logits;
  const float* temperature;  /* nullable [batch]; null: 1                   */
  const float* uniform;      /* [n_tokens]                                  */
  const float* noise;        /* [batch], row stride noise_stride            */
  int64_t noise_stride;
  int32_t* n_accepted;       /* out [batch]                                 */
  int32_t* out_tokens;       /* out [batch][max_out]: the accepted drafts,
                                the next token, then -1                     */
  float* logprobs;           /* out, nullable [batch][max_out]: log p of each
                                (0 when greedy and for -1)                  */
  int32_t* next_tokens;      /* out, nullable [batch]: the next token       */
  const int32_t* seq_lens;   /* nullable [batch]                            */
  int32_t* seq_lens_out;     /* out, nullable [batch], may be seq_lens:
                                seq_lens + n_accepted + 1 (unchanged for a
                                sequence without rows)                      */
} mpk_verify_args;

size_t mpk_verify_drafts_workspace(const mpk_token_batch* tok, int vocab);

/* One launch pair over the batch; see mpk_verify_args.  Float pointers need
 * 4-byte alignment only; d_workspace 256. */
mpk_status mpk_verify_drafts(const mpk_token_batch* tok,
                             const mpk_verify_args* args, void* d_workspace,
                             size_t workspace_bytes, uint32_t* d_status,
                             void* cuda_stream);

/* One step of drafted decoding of a whole model: the graph's rows are the
 * rows of *tok (so n_tokens is the batch that the graph was built for, and
 * tok->batch, at most as many, is the number of sequences), a sequence's
 * rows being its last accepted token and its drafts.  Runs the graph's
 * kernel-per-operator form (whatever its mode) with mpk_kv_append and
 * mpk_prefix_attention in the place of its attention, and mpk_verify_drafts
 * on the logits in the place of its argmax.  With one row a sequence, no
 * draft and T <= 0 it is mpk_decode_step over prefixes that are read once.
 *   v->tokens        the rows' input tokens, all in [0, vocab), those of
 *                    padding rows too
 *   v->logits        ignored, as are v->vocab, v->logits_stride and
 *                    v->seq_lens: the step's own (d_logits, fp32
 *                    [n_tokens][vocab], and kv->seq_lens)
 *   v->seq_lens_out  kv->seq_lens to keep the accepted tokens' keys and
 *                    values (those of the refused ones are overwritten by
 *                    the next step), null to leave the lengths alone
 * groups may be null.  Errors found on the device are those of the three
 * calls, in the graph's status word (mpk_get_status, mpk_reset).
 * MPK_ERR_UNSUPPORTED for the chained-linear mode. */
size_t mpk_verify_step_workspace(const mpk_graph* g,
                                 const mpk_token_batch* tok, int n_groups);
mpk_status mpk_verify_step(mpk_graph* g, const mpk_token_batch* tok,
                           const mpk_prefix_groups* groups,
                           const mpk_kv_cache* kv, const mpk_verify_args* v,
                           float* d_logits, void* d_workspace,
                           size_t workspace_bytes, void* cuda_stream);

#ifdef __cplusplus
}
#endif
#endif /* MPK_H_ */
