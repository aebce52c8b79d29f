/*
 * mg.h -- C ABI of the GB300 training-step library (libmg.so).
 *
 * One training step of a typed static graph -- forward pass, hand-derived
 * backward pass and optimizer update -- on one GPU, behind a fixed-shape plan.
 * The operation follows the Meganeura pages: "Meganeura" README, Example
 * section (a graph of input / parameter / matmul / relu / cross_entropy_loss
 * nodes, built once with build_session and stepped by a Trainer), Contents
 * section (SGD, Adam), Environment variables section (strict f32 scalar matmul
 * versus validated reduced-precision tiles); and the abstract of "Meganeura:
 * Portable GPU Training and Inference through Vulkan and Metal" (typed static
 * graph, automatic differentiation, optimizer, memory planner, runtime; strict
 * f32 kept apart from validated fast paths).
 *
 * Conventions for every call:
 *  - Pointers named params/grads/adam_m/adam_v/x/labels/out are DEVICE
 *    pointers owned by the caller (e.g. from torch tensors) and must be
 *    16-byte aligned.  The plan never frees them.
 *  - Everything is asynchronous on `stream` (a cudaStream_t; 0 = legacy
 *    default stream) except mg_loss, which synchronises it.
 *  - Every call returns an mg_status; nothing aborts, throws across the ABI or
 *    traps on the device.  mg_last_error() returns the message of the last
 *    failure (per plan, or process-wide for a NULL plan).
 *  - A plan is bound to the CUDA device that was current at creation and is not
 *    thread-safe: drive it from one host thread and one stream at a time.
 */
#ifndef MG_H
#define MG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mg_plan mg_plan;          /* opaque; owns the workspace */
typedef struct CUstream_st* mg_stream_t; /* same type as cudaStream_t */

typedef enum {
  MG_OK = 0,
  MG_ERR_INVALID_ARG = -1, /* NULL where a pointer is required, bad enum, bad value */
  MG_ERR_UNSUPPORTED = -2, /* a valid graph this library has no kernels for */
  MG_ERR_SHAPE = -3,       /* widths that do not chain, batch not a multiple of seq_len */
  MG_ERR_ALIGN = -4,       /* a pointer that is not 16-byte aligned */
  MG_ERR_OOM = -5,         /* workspace allocation failed (nothing leaked) */
  MG_ERR_CUDA = -6,        /* a CUDA runtime/driver error (launch or earlier async fault) */
  MG_ERR_NONFINITE = -7,   /* mg_debug_check_finite found a NaN or Inf */
  MG_ERR_TIMEOUT = -8,     /* a bounded device-side wait gave up */
  MG_ERR_INTERNAL = -9
} mg_status;

typedef enum {
  MG_OP_LINEAR = 0,           /* Y = X W (+ b), W[d_in, d_out] row-major, b[d_out] */
  MG_OP_RELU = 1,             /* max(z, 0); derivative 0 at z = 0 */
  MG_OP_GELU_TANH = 2,        /* 0.5 z (1 + tanh(sqrt(2/pi)(z + 0.044715 z^3))) */
  MG_OP_RMSNORM = 3,          /* y = x / sqrt(mean(x^2) + eps) * gamma, gamma[d] */
  MG_OP_RESIDUAL_BEGIN = 4,   /* remember the current value as the skip input */
  MG_OP_RESIDUAL_END = 5,     /* value = skip + value */
  MG_OP_CAUSAL_ATTENTION = 6, /* input [rows, 3d] = [Q|K|V], output [rows, d], d = n_heads*head_dim */
  MG_OP_EMBEDDING = 7,        /* first layer only: x is int32 ids [batch]; row = eps * W[id], W[d_in, d_out];
                                 an id outside [0, d_in) (padding): a row of zeros and no gradient */
  MG_OP_GROUPED_LINEAR = 8    /* Y[r] = X[r] W[e(r)], W[n_heads, d_in, d_out], the rows of group e given by
                                 mg_set_row_groups; rows of no group: zeros.  Activations and residual ends
                                 follow it as they follow LINEAR; no bias.  Strict forward sums are
                                 compensated, as LINEAR's */
} mg_op;

typedef enum { MG_LOSS_CE_DENSE = 0, MG_LOSS_CE_INDEX = 1, MG_LOSS_MSE = 2 } mg_loss_kind;
typedef enum { MG_PREC_STRICT_F32 = 0, MG_PREC_BF16 = 1 } mg_precision;
/* SGD: p -= lr g.  ADAM: bias-corrected moments, eps after the root.  LAPROP
 * (named beside Adam in the paper's checkpoint notes; the update is the
 * published LaProp algorithm): v = b2 v + (1-b2) g^2, m = b1 m + (1-b1) g /
 * (sqrt(v / (1 - b2^t)) + eps), p -= lr m / (1 - b1^t).  SGD_MOMENTUM:
 * heavy ball, b = beta1 b + g, p -= lr b (beta1 is the momentum). */
typedef enum {
  MG_OPT_SGD = 0,
  MG_OPT_ADAM = 1,
  MG_OPT_LAPROP = 2,
  MG_OPT_SGD_MOMENTUM = 3
} mg_optimizer;

typedef struct {
  int op;        /* mg_op */
  int d_in;      /* LINEAR, GROUPED_LINEAR: input width; RMSNORM: width; EMBEDDING: vocabulary */
  int d_out;     /* LINEAR, GROUPED_LINEAR: output width; EMBEDDING: width */
  int has_bias;  /* LINEAR: 1 if a bias vector follows W in the parameters */
  float eps;     /* RMSNORM: epsilon inside the square root; EMBEDDING: the rows' factor */
  int n_heads;   /* CAUSAL_ATTENTION; GROUPED_LINEAR: groups (at most 1024) */
  int head_dim;  /* CAUSAL_ATTENTION (64 supported) */
  int seq_len;   /* CAUSAL_ATTENTION: rows are [batch, seq_len] flattened */
} mg_layer;

typedef struct {
  int batch;               /* rows of x (tokens) */
  int n_layers;
  const mg_layer* layers;  /* copied at creation */
  int loss;                /* mg_loss_kind, applied to the last layer's output */
  int precision;           /* mg_precision */
  int optimizer;           /* mg_optimizer */
  float beta1, beta2, adam_eps;
} mg_graph_desc;

/* Build a plan for the current CUDA device: validate the descriptor, assign
 * parameter offsets, choose a kernel per GEMM, allocate the workspace once.
 * On failure *out is set to NULL and nothing is leaked.  The descriptor is the
 * typed static graph of the README's Example section, with its shapes fixed. */
mg_status mg_step_plan_create(const mg_graph_desc* desc, mg_plan** out);

/* Free the workspace.  NULL is a no-op.  Synchronises the device first.
 * (The session that build_session returns owns its device buffers for its
 * lifetime: "Meganeura" README, Example section.) */
void mg_step_plan_destroy(mg_plan* plan);

/* Floats in each of the flat parameter / gradient / moment buffers (the
 * parameter nodes of the README's Example section, packed). */
size_t mg_param_count(const mg_plan* plan);

/* Number of parameter tensors (W, b, gamma in declaration order): the graph's
 * parameter nodes ("Meganeura" README, Example section). */
int mg_param_tensor_count(const mg_plan* plan);

/* Tensor i of the flat buffers: element offset, logical rows and cols (a
 * vector has rows = 1).  Offsets are multiples of 64 elements; the gaps
 * between tensors are never read or written.  The logical shape is the one a
 * checkpoint stores, without device padding ("Meganeura" README, Contents
 * section, checkpoint notes). */
mg_status mg_param_info(const mg_plan* plan, int i, size_t* offset, int* rows, int* cols);

/* Bytes of device workspace the plan owns, after the memory planner's
 * lifetime sharing of gradient buffers (abstract of "Meganeura: Portable GPU
 * Training and Inference through Vulkan and Metal": memory planner; README,
 * Environment variables section: buffer lifetime aliasing, off with
 * MG_NO_ALIAS=1 here).  With MG_RECOMPUTE_GELU=1 at plan creation the GELU
 * pre-activations are not kept: the backward recomputes each one (the
 * forward's GEMM again, same inputs and weights, same result) into a single
 * shared buffer just before the input-gradient GEMM that needs it. */
size_t mg_workspace_bytes(const mg_plan* plan);

/* Forward pass only: the inference side of the train-to-deploy stack (README,
 * Contents section: a trained model reloaded into a fresh inference session;
 * abstract: one graph and runtime for training and deployed inference).
 * params: flat fp32 [mg_param_count]; x: [batch, d_in], fp32 in strict mode,
 * bf16 in bf16 mode (int32 ids [batch] for an embedding); out: fp32 [batch, d_out] (logits or the model output),
 * written row-major; in bf16 mode each output value is the bf16 value the
 * graph stores, widened. */
mg_status mg_forward(mg_plan* plan, const float* params, const void* x, float* out,
                     mg_stream_t stream);

/* One full training step: forward, loss, backward, optimizer update (README,
 * Example section: the Trainer's step over the session; Contents section: SGD
 * and Adam; abstract: automatic differentiation and optimizer).
 *  params  fp32 [P]  updated in place (fp32 master weights)
 *  grads   fp32 [P]  overwritten with dLoss/dparams of this step (before the update)
 *  adam_m, adam_v fp32 [P]  optimizer state, updated in place: Adam and LaProp
 *          use both (first and second moment); SGD_MOMENTUM keeps its velocity
 *          in adam_m (adam_v may be NULL); plain SGD needs neither
 *  x       [batch, d_in], fp32 (strict) or bf16 (bf16); int32 ids [batch] where
 *          the first layer is an embedding
 *  labels  CE_DENSE: fp32 [batch, C]; CE_INDEX: int32 [batch], values in [0, C);
 *          MSE: target [batch, d_out] in the activation dtype (fp32 / bf16)
 *  lr      learning rate; step: Adam's / LaProp's t, 1-based (ignored by SGD)
 * The loss of the step is kept on the device (mg_loss, mg_loss_device_ptr).
 * grads must not alias params.  The bf16 weight copy used by the bf16 path is
 * refreshed from params automatically when step == 1 or params differs from the
 * previous call; otherwise the previous update has kept it current.
 * Graph replay: the second call with the same six buffer addresses captures
 * the step's launches (both streams) into a CUDA graph, and that call and
 * later ones with those addresses launch the graph on `stream`, with lr and
 * the bias corrections of `step` written into its optimizer nodes.  Graphs
 * are kept for the two most recently used address sets (double-buffered
 * inputs).  Results are the same as launching each kernel.  Not used while
 * profiling or when `stream` is itself being captured; the environment
 * variable MG_GRAPH=0, read at plan creation, turns it off.  If a capture
 * fails the plan launches directly from then on.
 * With MG_FUSED_UPDATE=1 at plan creation (Adam, bf16) a weight whose
 * gradient GEMM runs on the tensor cores without a split over K is updated in
 * that GEMM's epilogue instead of the optimizer kernel: same results, one
 * launch fewer per such layer. */
mg_status mg_train_step(mg_plan* plan, float* params, float* grads, float* adam_m,
                        float* adam_v, const void* x, const void* labels, float lr, int step,
                        mg_stream_t stream);

/* Row groups of a plan's GROUPED_LINEAR layers (all have the same number of
 * groups): offsets [groups + 1] int32 in device memory, group e being the rows
 * offsets[e] .. offsets[e+1]-1; nondecreasing within [0, batch], clamped to
 * that where they are not.  The pointer is kept and its values are read on the
 * device by every mg_forward and mg_train_step from now on (write new values
 * to it, in stream order, as the batches change).  Required before either call
 * of a plan with such layers; a plan without them answers MG_ERR_INVALID_ARG. */
mg_status mg_set_row_groups(mg_plan* plan, const int* offsets);

/* Clip the gradients of every later mg_train_step by their global norm: with
 * norm = sqrt(sum of the squares of all gradients), the optimizer uses c * g, c
 * = max_norm / norm if norm > max_norm, else 1 (also for a norm that is NaN or
 * infinite).  `grads` still receives the gradients as they are, before the
 * factor.  max_norm = INFINITY measures only; 0 turns it off again (the state
 * after creation); anything else that is not positive is MG_ERR_INVALID_ARG.
 * With clipping on, the updates run after the whole backward instead of under
 * it (the sums of squares take their place there), and MG_FUSED_UPDATE has no
 * effect.  The first call that turns it on allocates 8 bytes per 2048
 * parameters.  Not while profiling. */
mg_status mg_set_grad_clip(mg_plan* plan, float max_norm);

/* Device address of {norm, c} (two fp32) of the last mg_train_step with
 * clipping on; NULL if it was never on.  Valid until destroy. */
const float* mg_grad_norm_device_ptr(const mg_plan* plan);

/* Copy {norm, c} to the host; synchronises `stream`. */
mg_status mg_grad_norm(mg_plan* plan, float* host_norm_and_factor, mg_stream_t stream);

/* Copy the last step's loss (the batch mean the README's Example section
 * prints per step) to the host; synchronises `stream`. */
mg_status mg_loss(mg_plan* plan, float* host_loss, mg_stream_t stream);

/* Enqueue, without waiting, a copy of the last step's loss and the plan's
 * pipeline error word to host memory: host_dst receives { float loss; int
 * timed_out; } (8 bytes; pinned memory keeps the copy asynchronous).  The
 * values are valid once `stream` has passed this point (an event, a later
 * synchronisation).  A nonzero timed_out means that step's results are
 * invalid; mg_loss reports it as MG_ERR_TIMEOUT and clears it.  For training
 * loops that enqueue the next step before reading this one's loss. */
mg_status mg_loss_async(mg_plan* plan, void* host_dst, mg_stream_t stream);

/* Device address of the last step's loss (one fp32, the batch mean of the
 * README's Example section), valid until destroy. */
const float* mg_loss_device_ptr(const mg_plan* plan);

/* Re-derive the bf16 weight copy from params (after the caller changed them,
 * e.g. a checkpoint restore).  A no-op in strict mode.  The copy is the
 * reduced-precision operand of the validated fast path, kept apart from the
 * strict f32 path (abstract; README, Environment variables section). */
mg_status mg_refresh_params(mg_plan* plan, const float* params, mg_stream_t stream);

/* ---- checkpoints --------------------------------------------------------
 * The paper's checkpoint notes: a checkpoint stores the logical tensors (no
 * device padding) and a restore is checked in full before it changes
 * anything.  Host-memory image, little-endian:
 *   64-byte header: magic "MGCKPT\0\1", u32 version (1), u32 tensor count,
 *     u32 flags (bit 0: first moment stored, bit 1: second moment stored),
 *     u32 precision of the saving plan, u64 values per section, u64 checksum
 *     of the sections, 24 reserved bytes;
 *   per tensor (mg_param_info order): u32 rows, u32 cols;
 *   sections, fp32: params, then the first moment, then the second moment,
 *     each the tensors' values back to back.
 * mg_checkpoint_bytes: the image size with the given sections.
 * mg_checkpoint_save: params (and m, v when non-NULL; v needs m) from the
 *   device into host_buf (cap bytes); *written gets the size; synchronises
 *   stream.  MG_ERR_INVALID_ARG when cap is too small.
 * mg_checkpoint_load: checks magic, version, tensor count and every shape
 *   against this plan, the size, the requested sections' presence and the
 *   checksum -- any failure returns an error with no device memory changed --
 *   then copies params (and m, v when non-NULL; moments stored but not asked
 *   for are skipped, e.g. when a forward-only or SGD plan takes a trained
 *   model) and refreshes the bf16 weight copy; synchronises stream.  The
 *   plan may differ from the saving one in everything but the tensors'
 *   shapes (precision, optimizer, batch). */
size_t mg_checkpoint_bytes(const mg_plan* plan, int with_m, int with_v);
mg_status mg_checkpoint_save(mg_plan* plan, const float* params, const float* m, const float* v,
                             void* host_buf, size_t cap, size_t* written, mg_stream_t stream);
mg_status mg_checkpoint_load(mg_plan* plan, const void* host_buf, size_t len, float* params,
                             float* m, float* v, mg_stream_t stream);

/* Human-readable schedule: one line per kernel with its shapes and the
 * workspace offsets: the dispatch order and alias map that the README's plan
 * dump switch prints at build (Environment variables section).  Writes at
 * most cap bytes including the terminating NUL; returns the full length. */
size_t mg_plan_dump(const mg_plan* plan, char* buf, size_t cap);

/* Message of the last failure; NULL plan gives the process-wide message.
 * (The pages have no counterpart: this is the ABI's error convention, in
 * place of the Rust API's panics and structured errors.) */
const char* mg_last_error(const mg_plan* plan);

/* Scan n floats (device) for NaN/Inf; synchronises stream.  Returns
 * MG_ERR_NONFINITE and the first bad index in *first_bad (may be NULL).  The
 * debug session's scan for the first NaN/Inf after a step ("Meganeura"
 * README, Debugging section). */
mg_status mg_debug_check_finite(mg_plan* plan, const float* data, size_t n, long long* first_bad,
                                mg_stream_t stream);

/* Kernels launched by the last mg_train_step / mg_forward call (a replayed
 * step counts the kernels its graph holds): the dispatch count of the
 * README's per-dispatch profile (Profiling section). */
int mg_last_launch_count(const mg_plan* plan);

/* mg_train_step calls served by a graph replay since the plan was created.
 * The step is compiled once and its fixed command list submitted every step
 * (README, Example section: build_session compiles once); here that list is
 * a CUDA graph. */
long long mg_graph_replays(const mg_plan* plan);

/* ---- per-kernel timing (CUDA events around each launch) ----------------
 * The per-dispatch timing profile of the README's Profiling section, with
 * CUDA events in place of hardware timestamp queries.
 * mg_profile_begin(plan, max_calls): from now on, each mg_train_step records
 * a start/stop event pair around every kernel, for up to max_calls calls.
 * mg_profile_end: synchronises, sums the elapsed time per schedule entry and
 * stops recording.  mg_profile_entry reads entry i (a kernel of the step):
 * its name, launches recorded, total milliseconds, and the algorithmic flops
 * and DRAM bytes of one launch. */
mg_status mg_profile_begin(mg_plan* plan, int max_calls);
mg_status mg_profile_end(mg_plan* plan);
int mg_profile_entries(const mg_plan* plan);
mg_status mg_profile_entry(const mg_plan* plan, int i, char* name, size_t name_cap,
                           int* launches, double* total_ms, double* flops, double* bytes);

/* ---- measurement ---------------------------------------------------------
 * The pages have no counterpart to this call: it measures the roofline
 * denominator of the strict-f32 path, whose matrix products run on the FP32
 * FFMA units only (the strict scalar matmul of the "Meganeura" README,
 * Environment variables section).  Runs a fused multiply-add kernel on every
 * SM of the current device for a few milliseconds, synchronises `stream`,
 * and writes the achieved FP32 TFLOP/s (2 flop per FFMA) to *tflops and the
 * same rate in flop per SM per clock of the device's maximum SM clock to
 * *flop_per_clk_per_sm (may be NULL; 0 if the clock rate is not reported).
 * It allocates and frees a few bytes of device memory. */
mg_status mg_ffma_peak(double* tflops, double* flop_per_clk_per_sm, mg_stream_t stream);

/* ---- softmax cross-entropy without device allocation -----------------
 * The Meganeura pages have no counterpart to this call.  It is for callers
 * that may not allocate device memory -- for example code running inside
 * another framework's plugin or kernel-enqueue hook, or a process whose device
 * memory is already reserved by its own caching allocator -- and therefore
 * cannot create a plan, whose workspace mg_step_plan_create allocates.
 *
 * Computes the same softmax cross-entropy loss and gradient as the training
 * step's loss kernel: for logits [rows, cols] row-major (dtype 0 = fp32,
 * 1 = bf16), labels dense fp32 [rows, cols] (label_kind 0) or int32 class ids
 * [rows] (label_kind 1), it writes dlogits (same dtype and layout as logits)
 * = (softmax * sum(y) - y) / rows and *loss (one fp32, device memory) = the
 * mean over rows of -sum_c y_c log softmax_c.  All pointers are caller-owned
 * device memory; nothing is allocated, and no cudaMalloc, cudaFree or
 * allocating library routine is called.
 *
 * Scratch: the per-row losses go to a fixed array in the library's device
 * memory of 65536 floats (256 KB), held by every GPU that loads the library
 * until the process exits.  rows above 65536 return MG_ERR_INVALID_ARG.  The
 * first call in each device context (the first call on a device, and the
 * first after a cudaDeviceReset re-creates the context) looks up that array's
 * device address with that device current; make that first call before any
 * stream capture.  All calls share the array: calls that overlap on the GPU
 * (different streams, or different host threads) race and give wrong results.
 * Each call overwrites the slots it reads, so nothing needs clearing between
 * calls.  A CUDA error already pending on the calling thread is returned as
 * MG_ERR_CUDA (the message says it came before the call) and nothing is
 * launched; launch failures carry the CUDA error string in the message. */
mg_status mg_softmax_ce_noalloc(int dtype, const void* logits, int rows, int cols, int label_kind,
                                const void* labels, void* dlogits, float* loss, mg_stream_t stream);

/* ---- language-model operators ---------------------------------------------
 * Calls that need no plan, for the ends of a language model's training step
 * and for serving; the layers `embedding` and `grouped linear` and
 * mg_set_grad_clip use the same kernels inside a plan.
 *
 * Conventions: dtype 0 = fp32, 1 = bf16.  Matrices are dense and row-major.
 * Pointers are caller-owned device memory of the current device, 16-byte
 * aligned (ids, offsets and gradient lists: to their element); a pointer of another
 * device or of pageable host memory is refused.  Everything is asynchronous on
 * `stream`, allocates nothing (mg_grad_list_create excepted), reads no value
 * back to the host, and can be captured into a CUDA graph.  A workspace is
 * scratch of one call at a time: calls that may overlap on the GPU (other
 * streams, other captured graphs) need one each.  Messages: mg_last_error(NULL).
 *
 * Embedding: out[i, :] = scale * table[ids[i], :], a product in fp32 rounded to
 * out's type.
 * id_kind 0 = int32, 1 = int64.  An id outside [0, vocab) -- padding -- reads
 * nothing: its row of out is 0.  table [vocab, dim], ids [n], out [n, dim];
 * n = 0 is allowed, dim is at most 2^30.
 *
 * Its gradient: dtable[v, :] = scale * sum over i with ids[i] == v of
 * dout[i, :], fp32 sums in ascending i order (long runs in a fixed order of
 * fixed windows), the same bits in every run.  All of dtable [vocab, dim]
 * fp32 is written, zeros for ids that do not occur; ids outside [0, vocab)
 * give nothing.  workspace: mg_embedding_workspace_bytes (for n ids or fewer; 0 for
 * arguments the call would refuse); its contents before the call do not matter. */
size_t mg_embedding_workspace_bytes(long long n, int vocab, int dim);
mg_status mg_embedding_forward(int table_dtype, const void* table, int vocab, int dim, int id_kind,
                               const void* ids, long long n, float scale, int out_dtype, void* out,
                               mg_stream_t stream);
mg_status mg_embedding_backward(int dtype, const void* dout, int vocab, int dim, int id_kind,
                                const void* ids, long long n, float scale, float* dtable,
                                void* workspace, size_t workspace_bytes, mg_stream_t stream);

/* Matrix products grouped by expert.  The rows of x [rows, d_in] are ordered
 * by group: group e has the rows offsets[e] .. offsets[e+1]-1, offsets
 * [groups + 1] int32 in device memory, nondecreasing within [0, rows] (values
 * that are not are clamped to that and never lead out of range).  Groups may
 * be empty and of any size.  w [groups, d_in, d_out].
 *   forward          y[r]  = x[r] w[e(r)]            [rows, d_out]
 *   backward_input   dx[r] = dy[r] w[e(r)]^T         [rows, d_in]
 *   backward_weight  dw[e] = x_e^T dy_e              [groups, d_in, d_out], fp32
 * dtype is the type of x, w, y, dx, dy; sums are fp32.  Rows outside
 * [offsets[0], offsets[groups]) and the weights of empty groups enter no result,
 * whatever they hold, and such rows are not written; dw of an empty group is 0.  groups at most 1024, rows and widths at most 2^30.  bf16 runs on
 * the tensor cores (rows of widths that are no multiples of 8 are copied to
 * aligned ones in the workspace first; small products of such widths, and fp32,
 * run on the CUDA cores).
 * workspace: mg_grouped_linear_workspace_bytes (for these rows or fewer); zero it
 * once before its first use.  Its first int is set to 1 if a bounded device-side wait gave up (never
 * seen), in which case that call's results are invalid; it stays 1 until the workspace is zeroed again.
 * mg_grouped_linear_status waits for `stream` and answers MG_ERR_TIMEOUT if it is set (not while
 * `stream` is being captured). */
size_t mg_grouped_linear_workspace_bytes(int rows, int groups, int d_in, int d_out);
mg_status mg_grouped_linear_forward(int dtype, const void* x, const int* offsets, int rows, int groups,
                                    int d_in, int d_out, const void* w, void* y, void* workspace,
                                    size_t workspace_bytes, mg_stream_t stream);
mg_status mg_grouped_linear_backward_input(int dtype, const void* dy, const int* offsets, int rows,
                                           int groups, int d_in, int d_out, const void* w, void* dx,
                                           void* workspace, size_t workspace_bytes,
                                           mg_stream_t stream);
mg_status mg_grouped_linear_backward_weight(int dtype, const void* x, const void* dy,
                                            const int* offsets, int rows, int groups, int d_in,
                                            int d_out, float* dw, void* workspace,
                                            size_t workspace_bytes, mg_stream_t stream);

mg_status mg_grouped_linear_status(const void* workspace, mg_stream_t stream);

/* Global gradient norm and clipping over many tensors.  A list holds n device
 * tensors (counts[i] elements of dtypes[i] at grads[i]) and where their scaled
 * values go: out[i], or in place where out is NULL or out[i] == grads[i].
 * Memory that is written may not overlap any other tensor of the list
 * (MG_ERR_INVALID_ARG).  counts[i] = 0 is allowed.  Creation copies the table
 * to the device and allocates 32 bytes per 32 KB of gradients; the list is
 * bound to the current device, and like a plan is used by one stream at a
 * time.
 * mg_grad_list_clip: stats[0] = norm = sqrt(sum of all squares), stats[1] =
 * c = max_norm / norm if norm > max_norm, else 1 (fp32, device memory, 8-byte
 * aligned; within a tensor of the list: MG_ERR_INVALID_ARG), and out = c * grads (c as rounded to
 * fp32: 0 where it is below 2^-150).  With c = 1 an in-place list is left as it
 * is.  A gradient that holds NaN or infinity gives such a norm and c = 1: the
 * gradients keep their bits for the caller to find.  (Finite gradients whose
 * norm is beyond fp32's range have stats[0] = infinity and are clipped.)
 * max_norm >= 0; INFINITY only measures.  A bounded device-side wait that gave
 * up (never seen) sets both stats to NaN, in that call and every later one of
 * the list; the outputs are then partly written.
 * (The wait of lists up to 15 MB: MG_CLIP_WAIT tries, read at creation.) */
typedef struct mg_grad_list mg_grad_list;
mg_status mg_grad_list_create(int n, const void* const* grads, void* const* out,
                              const size_t* counts, const int* dtypes, mg_grad_list** list);
void mg_grad_list_destroy(mg_grad_list* list);
mg_status mg_grad_list_clip(mg_grad_list* list, float max_norm, float* stats, mg_stream_t stream);

/* ---- log probabilities of tokens --------------------------------------------
 * Over each row x of logits [rows, vocab] (rows row_stride >= vocab elements
 * apart; pointers aligned to their element), with p = softmax(x / temperature):
 *   logp[r]     = log p[ids[r]]
 *   entropy[r]  = -sum_v p_v log p_v
 *   top_ids, top_logp [rows, k]: the k most likely tokens, most likely first, of
 *     equal ones the lowest first, and their log probabilities
 *   stats[r]    = {max x, log sum_v exp((x_v - max x) / temperature)}, for the
 *     backward
 * Each output may be NULL, but one (ids and logp are given together; k = 0: no
 * top_ids and top_logp).  k is at most MG_MAX_TOP and vocab.  fp32 sums; outputs
 * are fp32 and int32.
 * A row whose id is outside [0, vocab) -- padding -- enters nothing, whatever it holds:
 * its outputs are 0, its top_ids -1.  Logits of -inf have probability 0; a row of nothing else
 * has logp and top_logp -inf, entropy 0 and no gradient.  A row that holds a NaN
 * or +inf has NaN in logp, entropy and top_logp (its top_ids are in order, NaN
 * below -inf), and its gradient is NaN.
 *
 * backward: dlogits[r, v] = (dlogp[r] ([v = ids[r]] - p_v)
 *                            - dentropy[r] p_v (log p_v + entropy[r])) / temperature
 * with p from stats; dlogits has the logits' type and may be the logits
 * themselves (same rows), or lie in other columns of their buffer (same stride).
 * dlogp or dentropy may be NULL (no such gradient; entropy is not needed without
 * dentropy, ids without dlogp, unless there is padding).  Rows of padding, and rows
 * whose dlogp and dentropy are 0, are not read and get zeros.  Columns beyond vocab are
 * neither read nor written. */
#define MG_MAX_TOP 32
mg_status mg_token_logprobs(int dtype, const void* logits, long long rows, int vocab,
                            long long row_stride, int id_kind, const void* ids, float temperature,
                            float* logp, float* stats, float* entropy, int k, int* top_ids,
                            float* top_logp, mg_stream_t stream);
mg_status mg_token_logprobs_backward(int dtype, const void* logits, long long rows, int vocab,
                                     long long row_stride, int id_kind, const void* ids,
                                     float temperature, const float* stats, const float* entropy,
                                     const float* dlogp, const float* dentropy, void* dlogits,
                                     long long dlogits_stride, mg_stream_t stream);

/* ---- between two blocks of a residual network --------------------------------
 * From a block's output y and the residual stream x [rows, dim]:
 *   u     = y / sqrt(mean(y^2) + eps) * gamma_post     (u = y where gamma_post is NULL)
 *   x_out = scale x + gate * u                         (x_out = scale x + u where gate is NULL)
 *   h     = x_out / sqrt(mean(x_out^2) + eps) * gamma_pre   (not without h and gamma_pre)
 * gate [gates, dim]: each row of it for rows / gates consecutive rows (1: one
 * for all; rows: one each); gates = 0 without one.  dtype is the type of y, x,
 * x_out, h and their gradients; gammas, gate, their gradients and rstd [rows, 2]
 * (1 / sqrt of the two means, 1 where there is no norm; for the backward, may be
 * NULL) are fp32.  h is computed from x_out before its rounding.  Sums of squares
 * are fp32: finite within +-1e19 / sqrt(dim) (backward: those of gate gamma_post y x_out
 * too).
 * x_out and h may each be y or x itself.
 *
 * All pointers are 16-byte aligned, the vectors' too.
 *
 * backward, from dx_out and dh (either may be NULL, for none) and the forward's
 * inputs: dy, dx, and, where not NULL, dgamma_post, dgamma_pre [dim] and dgate
 * [gates, dim], fp32 sums in a fixed order (the same bits in every run).  dy and
 * dx may each be dx_out, dh, y or x itself.  Where y or x is not finite, that
 * element's dy and dx may be NaN without a norm too.  workspace:
 * mg_norm_residual_workspace_bytes (for these rows or fewer, of either type; 0 for
 * arguments the call would refuse); its contents before the call do not matter. */
size_t mg_norm_residual_workspace_bytes(int rows, int dim, int gates);
mg_status mg_norm_residual_forward(int dtype, const void* y, const void* x, int rows, int dim,
                                   const float* gamma_post, const float* gate, int gates,
                                   float scale, const float* gamma_pre, float eps, void* x_out,
                                   void* h, float* rstd, mg_stream_t stream);
mg_status mg_norm_residual_backward(int dtype, const void* dx_out, const void* dh, const void* y,
                                    const void* x, const float* rstd, int rows, int dim,
                                    const float* gamma_post, const float* gate, int gates,
                                    float scale, const float* gamma_pre, void* dy, void* dx,
                                    float* dgamma_post, float* dgate, float* dgamma_pre,
                                    void* workspace, size_t workspace_bytes, mg_stream_t stream);

/* ---- AdamW over many tensors ---------------------------------------------------
 * One step of every tensor of a list, with decoupled weight decay:
 *   g' = c grad;  m = beta1 m + (1 - beta1) g';  v = beta2 v + (1 - beta2) g'^2
 *   param = param (1 - lr weight_decay)
 *           - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 * (betas in [0, 1), eps a normal fp32 number.)
 * c = max_norm / norm[0] if norm[0] > max_norm, else 1; norm (device memory, may
 * be NULL: c = 1) is what mg_grad_list_clip with max_norm = INFINITY measures.
 * Where norm[0] is not finite the step changes nothing.
 * state_bits 32: m and v are fp32 [count].  state_bits 8: m and v are bytes
 * [count], the e4m3 codes of m and of sqrt(v), and m_scales, v_scales fp32
 * [ceil(count / 256)] the power of two that every 256 of them are multiplied by:
 * the least that keeps their largest finite magnitude at or below 446.72.  Zeros are
 * valid states.  Codes are rounded up or down at random with the probability of
 * the distance; the random bits depend on seed, step and the element's place in
 * the list alone, so that runs repeat bit for bit.  A moment that is not finite
 * becomes NaN, and leaves its neighbours as they are.
 * param is fp32 or bf16 (rounded to nearest), grad fp32 or bf16, copy (NULL, or
 * bf16 [count]) receives the rounded new parameters.  Pointers are aligned to
 * their element.  Memory that is written may not overlap any other of the list.
 * Creation copies the table to the device (80 bytes per 8192 elements, per 2048 of short
 * lists) and is bound to the current device; the list keeps no state of its own, but
 * a captured step reads the table and needs the list alive.
 * lr_device, step_device (device memory, fp32 and int32; NULL: lr and step are
 * taken) are read by the kernel, so that a captured step can be replayed with
 * new values; a step_device below 1 counts as 1.  Neither they nor norm may lie in
 * memory that the step writes. */
typedef struct {
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scales;    /* state_bits 8 */
  float* v_scales;
  void* copy;
  size_t count;       /* 0 is allowed */
  int param_dtype, grad_dtype;
  float weight_decay;
} mg_adamw_tensor;
typedef struct mg_adamw mg_adamw;
mg_status mg_adamw_create(int n, const mg_adamw_tensor* tensors, int state_bits, double beta1,
                          double beta2, double eps, unsigned long long seed, mg_adamw** opt);
void mg_adamw_destroy(mg_adamw* opt);
mg_status mg_adamw_step(mg_adamw* opt, double lr, long long step, const float* lr_device,
                        const int* step_device, const float* norm, float max_norm,
                        mg_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MG_H */
