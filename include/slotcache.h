/*
 * slotcache.h -- C ABI of the expert-slot MoE decode step for MI355X (gfx950).
 *
 * One MoE layer of an expert-offloaded mixture-of-experts model keeps S fixed
 * HBM slots, each able to hold one routed expert; every expert of the layer
 * lives in a pinned host backing store, and the slots are an LRU cache over
 * it.  One decode step (moe_layer_decode) runs, all on the device and all
 * enqueued on the caller's stream:
 *   router top-k -> expert id to slot remap with LRU victim choice -> copy of
 *   missed experts' weight and scale rows from host into their victim slots ->
 *   routed gate/up and down products on NVFP4 weights with SiLU -> weighted
 *   top-k combine.
 * The method is the slot cache of the page "GLM 5.3 Testing: HBM Expert
 * Allocation" (sections "What the slot cache is" and "The build, measured on a
 * synthetic GLM-shaped layer"), with the LRU occupancy of the page "GB300 GLM
 * 5.3 Testing" (section "Expert allocation vs a cache").
 *
 * Conventions.
 *  - Every call returns sc_status: SC_OK (0) or a negative error; nothing
 *    aborts or throws.  slotcache_last_error() gives a message for the last
 *    non-OK status on the calling thread.
 *  - Pointers named d_* are device pointers (hipMalloc / torch CUDA tensors);
 *    pointers named h_* or host_* are host pointers.  `stream` is a
 *    hipStream_t passed as void* (NULL = the null stream).
 *  - The caller owns every device buffer (slot pool, state, workspace,
 *    logits, x, y) and the stream.  The library owns the pinned host backing
 *    store (allocated at the exact size, no power-of-two rounding) and frees
 *    it in slotcache_destroy.
 *  - Calls that use one handle must be ordered: the same stream, or streams
 *    the caller synchronizes.  They share one workspace.
 *
 * Data formats (one expert "blob", B_e bytes; the same layout in a slot and in
 * the backing store):
 *   [w13 codes  2I x H/2 bytes] rows 0..I-1 gate, rows I..2I-1 up
 *   [w13 scales 2I x H/16     ] one FP8 E4M3 (OCP "FN") per 16 K-elements
 *   [w2 codes   H x I/2       ]
 *   [w2 scales  H x I/16      ]
 *   Codes are FP4 E2M1, two per byte, the even element in the low nibble.
 *   Element value = e2m1(code) * e4m3(block scale) * global scale, with one
 *   fp32 global scale per (expert, matrix) held in a device table.
 *   B_e = 27*H*I/16 (21,233,664 B for H=6144, I=2048).
 */
#ifndef SLOTCACHE_H
#define SLOTCACHE_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__) || defined(__clang__)
#define SC_API __attribute__((visibility("default")))
#else
#define SC_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SC_OK = 0,
  SC_E_ARG = -1,          /* invalid argument or configuration; nothing enqueued */
  SC_E_HOST_OOM = -2,     /* pinned host allocation failed */
  SC_E_HIP = -3,          /* a HIP runtime call failed */
  SC_E_STATE = -4,        /* call not valid in the handle's state */
  SC_E_DEVICE = -5,       /* a device-side check latched an error word */
  SC_E_UNSUPPORTED = -6   /* shape outside the compiled kernel set */
} sc_status;

typedef struct sc_handle sc_handle;

/* Rows per step above which a step always reads the backing store directly
 * (the prefill bypass; page "GLM 5.3 Testing: HBM Expert Allocation", section
 * "What the slot cache is"). */
#define SC_BYPASS_ROWS 16

typedef struct {
  int32_t n_layers;               /* >= 1 */
  int32_t hidden;                 /* H: 256, 512, 1024, 2048, 4096, 6144 or 8192 */
  int32_t inter;                  /* I: 128 ... 8192 (same set plus 128) */
  int32_t n_experts;              /* E: top_k <= E <= 1024 */
  int32_t top_k;                  /* k: 1 <= k <= 32 */
  const int32_t* slots_per_layer; /* host [n_layers]; 1 <= S_l <= min(E, 1024) */
  int32_t max_rows;               /* largest M the caller will pass, 1..256 */
  int32_t n_banks;                /* host backing banks, 1..n_layers; layer l reads bank l % n_banks */
  int32_t event_capacity;         /* per-layer miss-event ring, records (0 = 4096) */
  uint32_t flags;                 /* 0, or SC_FLAG_BATCH_INVARIANT and/or SC_FLAG_OVERLAP_FILL */
  int32_t prefill_stage;          /* G, experts staged per prefill group, 0..1024 (see below) */
} sc_config;

/* Prefill groups.  A step of more than SC_BYPASS_ROWS rows (a prefill chunk)
 * always bypasses the cache.  With prefill_stage = 0 its non-resident experts
 * are read in place from the host-mapped backing store by the expert kernels.
 * With G = prefill_stage > 0 the workspace holds a G-blob staging area in HBM:
 * the step's non-resident experts, in first-occurrence order, are copied into
 * it G at a time by the fill kernel, and each group's expert products (the
 * resident experts go with the first group) run from HBM before the next
 * group is copied; the weighted combine runs once, after the last group, so
 * the output is the same bits as without staging.  The pages' prefill-groups
 * knob stages 64 experts at a time and reduces once (page "glm53 -
 * GLM-5.3-Flash (NVFP4)").  A step of M rows enqueues ceil(min(M*k, E) / G)
 * groups; groups left empty exit at once.  Ignored (no staging area) when
 * max_rows <= SC_BYPASS_ROWS. */

/* Every row of a step computes the bits it would compute alone, as a one-row
 * step: the streaming FP4 kernels run for every M (their per-row reduction
 * order does not depend on how many rows share an expert) and the matrix-core
 * kernels, whose rounding differs, are not used.  Drafted and verify rows then
 * never change a row's output (the exact-decoding rule on the page "TensorFold
 * GLM-5.3 explained").  Costs speed from M = 5 on (the matrix-core ranges
 * below). */
#define SC_FLAG_BATCH_INVARIANT 1u

/* Overlapped miss fill for one-row steps (M = 1).  The copy of the step's
 * misses into their slots shares one launch with the gate/up products of the
 * experts it does not write, which run while the copy crosses the host link;
 * the copied experts' gate/up follows, then down and the combine.  The pages
 * name asynchronous miss fills as what could take the copy off the critical
 * path (page "GB300 GLM 5.3 Testing", September 13 update of the section
 * "Speculation: what is holding the GB300 back, and what probably wins
 * next").  Outputs, slots and bookkeeping are the same bits as without the
 * flag.  The trade-off: a step with misses finishes sooner by about the
 * resident experts' gate/up time, but the copy blocks take wave slots from
 * the products, so an all-hit step's gate/up runs slower.  Steps of more than
 * one row are not affected.  With events (moe_layer_decode_ev) both the
 * fill and the gate/up events bracket the shared launch; the fill spans are
 * those of its copy blocks and the gate/up spans those of its product blocks
 * (slotcache_read_kernel_spans); the copied experts' gate/up launch is not
 * timed. */
#define SC_FLAG_OVERLAP_FILL 2u

/* Without SC_FLAG_BATCH_INVARIANT, steps of at least this many rows run the
 * gate/up (resp. down) product on the matrix cores; their rows need not be
 * bit-equal to the same rows decoded alone (the outputs stay within the same
 * tolerance of the exact result).  Below them the streaming kernels run, whose
 * rows are bit-equal to one-row steps: on steps of 2 to 4 rows both products
 * keep the expert's pick operands in LDS and widen each weight once for all
 * of them. */
#define SC_MFMA_MIN_ROWS_GATEUP 5
#define SC_MFMA_MIN_ROWS_DOWN 5

typedef struct {
  size_t blob_bytes;              /* B_e */
  size_t slot_pool_bytes;         /* device: sum over layers of S_l * B_e; 256-B aligned base */
  size_t state_bytes;             /* device: maps, LRU keys, counters, event rings, global scales */
  size_t workspace_bytes;         /* device: per-call scratch shared by all layers, with the
                                     prefill staging area (G * B_e) when there is one */
  size_t backing_bytes_per_bank;  /* host, allocated by the library: E * B_e */
} sc_sizes;

typedef struct {
  uint64_t steps;         /* calls of moe_layer_decode on the layer */
  uint64_t bypass_steps;  /* steps that read the backing store directly */
  uint64_t picks;         /* M*k over cached steps */
  uint64_t lookups;       /* unique experts over cached steps */
  uint64_t hits;          /* unique experts already resident */
  uint64_t misses;        /* unique experts copied into a slot */
  uint64_t evictions;     /* misses whose victim slot held an expert */
  uint64_t bytes_filled;  /* misses * B_e, host to HBM */
  uint64_t bypass_bytes;  /* unique experts * B_e read from host by bypass steps */
  uint32_t device_error;  /* nonzero: a device-side bounds check failed */
  uint32_t reserved;
} sc_stats;

typedef struct {
  int64_t step;     /* value of the layer's step counter when the miss happened */
  int32_t expert;   /* expert copied in */
  int32_t slot;     /* its slot */
  int32_t evicted;  /* expert that held the slot, or -1 for an empty slot */
  int32_t reserved;
} sc_event;

/* Sizes of the device buffers the caller must allocate for `cfg`, so that every
 * device buffer is sized once, up front, before any step runs.  The pages lost
 * launches to memory that was taken after the budget had been set (page "glm53 -
 * GLM-5.3-Flash (NVFP4)", section "Context and the KV cap": a cache allocated
 * after the framework's memory profiling) and to budgets checked in the wrong
 * units (page "GLM 5.3 Testing: HBM Expert Allocation", section "Five launches,
 * four failures").  Byte counts are exact (no rounding to a power of two).
 * Pure: no device or host allocation.  SC_E_ARG / SC_E_UNSUPPORTED for an
 * invalid or unsupported configuration; *out is left untouched then. */
SC_API sc_status slotcache_query_sizes(const sc_config* cfg, sc_sizes* out);

/* Binds caller-allocated device buffers (sizes from slotcache_query_sizes,
 * 256-byte aligned), allocates the pinned backing store (n_banks * E * B_e
 * bytes, exact size, device-mapped) and resets every layer to the cold state:
 * all slots empty, keys -1, counters zero, global scales 1.0.  Synchronous.
 * The device buffers must outlive the handle.
 * Page "GLM 5.3 Testing: HBM Expert Allocation": the per-layer slots and the
 * pinned backing store are section "What the slot cache is"; pinning at the
 * exact byte size (a rounding pinned allocator wasted a third of host memory)
 * is section "Five launches, four failures"; the cache starts empty and is
 * filled on demand (page "TensorFold GLM-5.3 explained": nothing is resident
 * for good).  Errors: SC_E_ARG (bad config, NULL or misaligned buffer),
 * SC_E_HOST_OOM (pinned allocation failed; nothing is kept), SC_E_HIP; *out is
 * NULL on any error. */
SC_API sc_status slotcache_init(const sc_config* cfg, void* d_slot_pool, void* d_state,
                         void* d_workspace, sc_handle** out);

/* Host pointer and size of backing bank `bank` ([E][B_e] blobs, expert-major).
 * The caller fills it before the first step that reads it and must not write
 * it while steps are in flight. */
SC_API sc_status slotcache_backing(sc_handle* h, int32_t bank, void** host_ptr, size_t* bytes);

/* Copies the fp32 global scales of bank `bank` from host memory h_gs[E][2]
 * ((w13, w2) per expert) to the device table.  Synchronous. */
SC_API sc_status slotcache_set_global_scales(sc_handle* h, int32_t bank, const float* h_gs);

/* Warm start for `layer`: slot s <- expert s for s < S (copied from the
 * backing store), keys -1, no pinned slots.  Synchronous.  With S == E this
 * makes every expert resident (the all-resident layer). */
SC_API sc_status slotcache_preload(sc_handle* h, int32_t layer);

/* One decode step of `layer` for M rows (1 <= M <= max_rows), the method of
 * page "GLM 5.3 Testing: HBM Expert Allocation", section "What the slot cache
 * is" (ids mapped to slots on the device before the expert launch, misses copied
 * into LRU victims, the expert products reading the same bytes as with every
 * expert resident, more than 16 rows bypassing, fixed addresses and shapes for
 * graph capture), with the fp32 combine of its section "A correction first":
 *   d_logits fp32 [M][E], d_x bf16 bits [M][H], d_y fp32 [M][H] (written).
 * Router: per row the k largest logits (ties -> lower expert id, NaN below
 * -inf), weights = softmax over the k chosen logits.  Cached steps (M <= 16
 * and at most S unique experts, see slotcache_pin for pinned slots) remap,
 * fill misses and compute from the slots; other steps (bypass) leave the cache
 * untouched and compute resident experts from their slots and the others from
 * the backing store.  Asynchronous on `stream`, no host synchronisation and no
 * allocation, so it can be captured into a HIP graph (fixed addresses and
 * shapes).  Argument errors return before anything is enqueued. */
SC_API sc_status moe_layer_decode(sc_handle* h, int32_t layer, const float* d_logits,
                           const uint16_t* d_x, int32_t M, float* d_y, void* stream);

/* Bytes of the library's static per-call scratch on each GPU (see
 * moe_layer_decode_static). */
#define SC_STATIC_SCRATCH_BYTES 16777216

/* moe_layer_decode for callers that cannot allocate: code under HIP graph
 * capture that must not touch an allocator, tight serving loops, harnesses
 * that forbid allocation.  The step's per-call scratch (routing lists, pick
 * grouping, h, per-pick down outputs) comes from a fixed device array of the
 * library, SC_STATIC_SCRATCH_BYTES per GPU, set up by slotcache_init on the
 * handle's device and held until the process ends, instead of the workspace
 * bound to the handle.  The caller still passes logits, x and y, and the
 * handle's slots and state are used as by moe_layer_decode; the results are
 * the same bits.  The call allocates nothing, host or device.
 * Every call on a GPU shares that GPU's array and leaves its contents behind
 * (each step writes every scratch word it reads before reading it, so nothing
 * needs clearing): calls that can overlap on one GPU -- streams not ordered
 * with each other, from this or any other handle -- race on it and must not
 * be issued.  slotcache_read_routing reads the array after such a step.
 * Errors (SC_E_ARG, nothing enqueued): the arguments of moe_layer_decode;
 * M > SC_BYPASS_ROWS (a prefill chunk needs the caller's workspace and its
 * staging area); a configuration whose per-call scratch for
 * min(max_rows, SC_BYPASS_ROWS) rows exceeds SC_STATIC_SCRATCH_BYTES (the
 * message gives both sizes); the array could not be set up at init. */
SC_API sc_status moe_layer_decode_static(sc_handle* h, int32_t layer, const float* d_logits,
                                         const uint16_t* d_x, int32_t M, float* d_y, void* stream);

/* Kernels of one step, for per-kernel timing: routing+remap, miss fill,
 * gate/up, down, combine. */
#define SC_N_KERNELS 5
#define SC_N_EVENTS (2 * SC_N_KERNELS)
/* moe_layer_decode with per-kernel timing: events[2i] and events[2i+1]
 * (hipEvent_t passed as void*, created by the caller) are stamped at the start
 * and the end of kernel i's execution (hipExtLaunchKernelGGL).  On a staged
 * prefill step the fill, gate/up and down events and spans are those of the
 * first group's launches.  events == NULL is moe_layer_decode. */
SC_API sc_status moe_layer_decode_ev(sc_handle* h, int32_t layer, const float* d_logits,
                              const uint16_t* d_x, int32_t M, float* d_y, void* stream,
                              void* const* events);

/* Pins experts of `layer` (hybrid policy: page "GB300 GLM 5.3 Testing",
 * section "Expert allocation vs a cache", compares a static pin with LRU):
 * slot i <- h_experts[i] for i < n (copied from the backing store), never a
 * victim; LRU runs over the other S - n slots, which are emptied (keys -1).
 * 0 <= n <= S distinct ids; n = 0 unpins.  The step counter and counters are
 * kept.  With n pinned slots a step bypasses when its unique experts outside
 * the pinned set exceed S - n (the rule |U| > S for n = 0); n = S is a static
 * pin.  slotcache_preload clears the pins; slotcache_write_state requires the
 * pinned slots to keep their experts.  Synchronous. */
SC_API sc_status slotcache_pin(sc_handle* h, int32_t layer, const int32_t* h_experts, int32_t n);

/* Execution spans of the kernels of the most recent step run through
 * moe_layer_decode_ev, in microseconds: us_out[i] (i < SC_N_KERNELS) is the
 * time from kernel i's first block start to its last wavefront end, read from
 * stamps the kernels write with the device's constant wall clock.  (The stop
 * events of hipExtLaunchKernelGGL land a few microseconds after a kernel's
 * end, which matters for kernels of tens of microseconds.)  Synchronizes the
 * stream of the last step.  SC_E_STATE if that step was not a timed one. */
SC_API sc_status slotcache_read_kernel_spans(sc_handle* h, double* us_out);

/* Counters of `layer`: the hit and miss counts that the pages read from the
 * engine's periodic cache statistics (page "GB300 GLM 5.3 Testing", section
 * "Sizing the context window: 256K, measured") and keep as hit/miss logs beside
 * every speed claim (same page, section "What changed in our policy").
 * Synchronizes the stream of the last step.  SC_E_DEVICE (with *out filled) when
 * a device-side check latched an error word on the layer. */
SC_API sc_status slotcache_stats(sc_handle* h, int32_t layer, sc_stats* out);

/* Slot map and LRU clock of `layer` (synchronizes): h_e2s int32[E] (slot or
 * -1), h_s2e int32[S] (expert or -1), h_key int64[S] (-1 = empty), h_step
 * (step counter).  Any output pointer may be NULL.  The slots are only a cache:
 * the backing store keeps the only full copy of every expert (page "TensorFold
 * GLM-5.3 explained"), so this state plus the backing store is a complete
 * checkpoint of the layer, and it is what the pages' "no stale slots" parity
 * check inspects (page "GB300 GLM 5.3 Testing", section "What changed in our
 * policy"). */
SC_API sc_status slotcache_read_state(sc_handle* h, int32_t layer, int32_t* h_e2s, int32_t* h_s2e,
                               int64_t* h_key, int64_t* h_step);

/* Restores a state read by slotcache_read_state (checkpoint / resume; the
 * backing store keeps the only full copy, page "TensorFold GLM-5.3 explained"):
 * copies the resident experts' blobs from the backing store into their slots
 * and writes maps, keys and step counter.  Counters and the event ring are left
 * as they are.  Synchronous.  SC_E_ARG, with nothing written, unless: the maps
 * are mutually inverse; empty slots have key -1; every occupied slot's key is a
 * clock value the layer could have stamped, -1 <= key < step * 16 * k (-1: never
 * referenced since it was filled); 0 <= step < 2^40; pinned slots keep their
 * experts. */
SC_API sc_status slotcache_write_state(sc_handle* h, int32_t layer, const int32_t* h_e2s,
                                const int32_t* h_s2e, const int64_t* h_key, int64_t step);

/* Miss events of `layer`, oldest first (synchronizes): the per-miss record
 * (step, expert in, slot, expert evicted) behind the pages' hit/miss logs (page
 * "GB300 GLM 5.3 Testing", section "What changed in our policy") and their
 * bit-exact churn comparisons (page "GLM 5.3 Testing: HBM Expert Allocation",
 * section "The build").  Copies up to `cap` records of the most recent
 * min(total, event_capacity) into h_buf; *n_out = records copied, *total =
 * events ever logged (total > event_capacity means the ring wrapped).  SC_E_ARG
 * if h_buf is NULL while records are available and cap > 0. */
SC_API sc_status slotcache_read_events(sc_handle* h, int32_t layer, sc_event* h_buf, size_t cap,
                                size_t* n_out, uint64_t* total);

/* Routing of the most recent step (synchronizes): h_ids int32[M*k],
 * h_w fp32[M*k] in (row, rank) order, *M_out = M, *bypass = 1 if the step
 * bypassed the cache.  Outputs may be NULL. */
SC_API sc_status slotcache_read_routing(sc_handle* h, int32_t* h_ids, float* h_w, int32_t* M_out,
                                 int32_t* bypass);

/* ---- 4-bit weights -------------------------------------------------------- */

/* Element types of dense tensors. */
#define SC_DTYPE_F32 0
#define SC_DTYPE_BF16 1
#define SC_DTYPE_F16 2

/* 4-bit weight formats: E2M1 codes, two per byte, the even element in the low
 * nibble, with a scale per group of consecutive elements of a row.
 *   SC_FP4_NV  one E4M3 scale per 16 elements and one fp32 scale of the matrix
 *              (the format of the expert blobs)
 *   SC_FP4_MX  one E8M0 scale (2^(byte - 127), 255 is NaN) per 32 elements */
#define SC_FP4_NV 0
#define SC_FP4_MX 1

/* A matrix [rows][cols] held in 4 bits, in device memory.  cols is a multiple
 * of the group; rows follow each other without padding. */
typedef struct {
  int32_t format;          /* SC_FP4_NV or SC_FP4_MX */
  int32_t rows;            /* >= 0 */
  int32_t cols;            /* <= 2^20; rows * cols <= 2^36 - 16 */
  void* d_codes;           /* [rows][cols/2], 16-byte aligned */
  void* d_scales;          /* [rows][cols/16] or [rows][cols/32], 2-byte aligned */
  float* d_global_scale;   /* one float; NULL stands for 1 where it is only read */
} sc_fp4_matrix;

#define SC_FP4_QUANT_WORKSPACE_BYTES 4096

/* Quantises d_w [rows][cols] (row stride ldw elements, type w_type) into `out`.
 * NVFP4: the matrix scale is read from out->d_global_scale when scale_given is
 * nonzero (positive and finite; matrices that share one, or a gate/up pair cut
 * into shards), else it is max|w| / 2688 and written there (1 when that is 0).
 * A group's scale is the E4M3 number nearest to max|group| / (6 scale), at most
 * 448; a code is the E2M1 number nearest to w / (group scale * scale), at most
 * 6.  MXFP4: the group scale is 2^(floor(log2 max|group|) - 2).  Nearest is of
 * the exact quotient, ties to even.  A group whose scale rounds to 0 has codes
 * 0.  Infinities and NaN do not count in the matrix scale; a group that holds
 * one gets a NaN scale, so that it reads back as NaN.  d_workspace:
 * SC_FP4_QUANT_WORKSPACE_BYTES of device memory when the scale is computed
 * (NVFP4 without scale_given), else ignored.  Asynchronous on `stream`, whose
 * device is current; can be captured.  rows == 0 does nothing. */
SC_API sc_status fp4_quantize(const void* d_w, int32_t w_type, int64_t ldw, const sc_fp4_matrix* out,
                              int32_t scale_given, void* d_workspace, void* stream);

/* Writes the values `w` stands for to d_w (type w_type, row stride ldw): code *
 * group scale * matrix scale, rounded to fp32 once and then to w_type. */
SC_API sc_status fp4_dequantize(const sc_fp4_matrix* w, void* d_w, int32_t w_type, int64_t ldw, void* stream);

/* y = x W^T + bias: x [M][w->cols] of bf16 or fp16 (row stride ldx elements), y
 * [M][w->rows] (row stride ldy, type y_type), bias fp32 [w->rows] or NULL.
 * Products of x with the codes (up to 4 rows) or with the codes times their group
 * scales (more rows) are exact, sums are fp32, and y is rounded once.  For the
 * sums to be finite |x| has to stay below 2^121, and a code times its group scale
 * below 2^128, as every matrix from fp4_quantize has it.  Any M >= 0; a NaN or
 * infinity in a row of x or of W stays in its row or column of y.  y must not overlap
 * x or the weights.  Asynchronous on `stream`, whose device is current; no
 * workspace, no allocation; can be captured. */
SC_API sc_status fp4_linear(const sc_fp4_matrix* w, const void* d_x, int32_t x_type, int64_t ldx, int32_t M,
                            const float* d_bias, void* d_y, int32_t y_type, int64_t ldy, void* stream);

/* ---- a whole MoE layer for a few tokens --------------------------------------- */

#define SC_MOE_MAX_ROWS 16

/* How router logits become picks and weights.  Both pick the k largest (ties
 * to the lower expert id, NaN lowest) and multiply the weights by routed_scale.
 *   SC_SCORE_SOFTMAX  picks by logit; weights are the softmax over the k chosen
 *                     logits (the rule of moe_layer_decode)
 *   SC_SCORE_SIGMOID  picks by sigmoid(logit) + bias (compared in fp64, so that
 *                     scores near 1 stay apart; without a bias by the logit);
 *                     weights are the chosen sigmoids divided by their sum
 *                     (equal when that is 0) */
#define SC_SCORE_SOFTMAX 0
#define SC_SCORE_SIGMOID 1

typedef struct {
  int32_t hidden;          /* H: a multiple of 64 in [64, 32768] */
  int32_t inter;           /* I: a multiple of 64 in [64, 32768] */
  int32_t n_experts;       /* top_k <= E <= 1024 */
  int32_t top_k;           /* 1 <= k <= 32 */
  int32_t shared_inter;    /* inner size of the shared expert, 0 for none, else as I */
  int32_t max_rows;        /* largest M of a call, 1 .. SC_MOE_MAX_ROWS */
  int32_t score;           /* SC_SCORE_SOFTMAX or SC_SCORE_SIGMOID */
  float routed_scale;      /* factor of the routed experts' sum */
} sc_moe_config;

typedef struct {
  const void* d_router;            /* bf16 [E][H], 16-byte aligned */
  const float* d_score_bias;       /* fp32 [E] or NULL; only SC_SCORE_SIGMOID uses it */
  const void* d_blobs;             /* [E][B_e] expert blobs in HBM, 16-byte aligned: a full slot pool, or a copy */
  const float* d_global_scales;    /* fp32 [E][2] (w13, w2) */
  const void* d_shared_blob;       /* the shared expert as a blob of its own inner size, 16-byte aligned */
  const float* d_shared_scales;    /* fp32 [2] */
} sc_moe_weights;

/* Bytes of device workspace that moe_layer_forward needs. */
SC_API sc_status moe_layer_workspace_bytes(const sc_moe_config* cfg, size_t* bytes);

/* Enqueues the clearing of a workspace's control words (256-byte aligned), whose
 * places follow from the configuration: once per workspace and configuration,
 * max_rows included, before the first forward call with it; not needed between
 * calls.  Also after forward calls that ran on one workspace without being
 * ordered, once all of them are done. */
SC_API sc_status moe_layer_prepare(const sc_moe_config* cfg, void* d_workspace, void* stream);

/* One layer for M rows of x (bf16 [M][H], row stride ldx): y [M][H] (fp32 or
 * bf16, row stride ldy) = sum over the row's k picks of weight * D(silu(G x) *
 * (U x)), plus the shared expert's output.  d_ids int32 [M][k] and d_weights
 * fp32 [M][k] receive the picks in rank order (either may be NULL).  Products
 * are exact, sums fp32, the order of every sum is fixed; y is rounded once.  A
 * row's result does not depend on the other rows beyond rounding, and not at
 * all when it holds a NaN.  M == 0 does nothing.  Asynchronous on `stream`,
 * whose device is current; no allocation; can be captured.  Calls that share a
 * workspace must be ordered (one stream, or streams that the caller orders);
 * y must not overlap x.  Blocks wait for each other's results; a wait that lasts
 * over a second (only calls that break that order can do this) gives the call up: y
 * is NaN then, d_ids and d_weights are undefined, and the control words are as
 * after moe_layer_prepare unless the other call changed them since. */
SC_API sc_status moe_layer_forward(const sc_moe_config* cfg, const sc_moe_weights* w, void* d_workspace,
                                   const uint16_t* d_x, int64_t ldx, int32_t M, void* d_y, int32_t y_type,
                                   int64_t ldy, int32_t* d_ids, float* d_weights, void* stream);

/* ---- attention over prompts ------------------------------------------------- */

#define SC_PROMPT_MAX_HEADS 1024
#define SC_PROMPT_MAX_SEQS 65536
#define SC_PROMPT_MAX_ROWS (1 << 24)
#define SC_PROMPT_MAX_STRIDE (1 << 23)   /* elements from a key or value to the next */

#define SC_PROMPT_PART_KEYS 2048
#define SC_ATTENTION_MAX_SCALE 2.3e38f   /* times log2 e it is still an fp32 number */

/* Packed sequences: sequence b has the rows d_starts[b] .. d_starts[b+1]-1 of q
 * and the keys d_key_starts[b] .. d_key_starts[b+1]-1 of k and v.  Element d of
 * row t and head h of q is at t * q_stride[0] + h * q_stride[1] + d, and so for
 * k, v and out (strides in elements). */
typedef struct {
  int32_t type;                   /* of q, k, v and out: SC_DTYPE_BF16 or SC_DTYPE_F16 */
  int32_t head_dim;               /* 64, 128 or 256 */
  int32_t q_heads, kv_heads;      /* q_heads is a multiple of kv_heads; head h reads key head h / (q_heads / kv_heads) */
  int32_t n_seqs;                 /* <= SC_PROMPT_MAX_SEQS */
  int32_t rows, keys;             /* of all sequences; (rows / 128 + n_seqs) * q_heads < 2^24 */
  float scale;                    /* > 0, <= SC_ATTENTION_MAX_SCALE */
  const void* d_q;
  const void* d_k;
  const void* d_v;
  void* d_out;
  float* d_lse;                   /* [rows][q_heads] or NULL */
  const int32_t* d_starts;        /* [n_seqs + 1] */
  const int32_t* d_key_starts;    /* [n_seqs + 1]; d_starts for whole prompts */
  int64_t q_stride[2], k_stride[2], v_stride[2], out_stride[2];
} sc_prompt;

/* Bytes of device workspace that prompt_attention needs: 0 but where few blocks of
 * rows, or blocks of uneven lengths, have many keys (2 * SC_PROMPT_PART_KEYS per
 * sequence and more), and at most 5120 * 128 * (4 * head_dim + 8).  Reads the sizes only. */
SC_API sc_status prompt_attention_workspace_bytes(const sc_prompt* p, size_t* bytes);

/* Causal attention of every row over its sequence's keys: with Lq rows and Lk
 * keys row i sees the keys below Lk - Lq + i + 1.  out = softmax(scale q k^T) v
 * of the keys seen, lse the natural logarithm of the sum of exponentials; a row
 * that sees none gets 0 and -infinity.  Products are exact, sums and softmax
 * statistics fp32, P is rounded to the type of v, out once.  Rows outside of the
 * sequences are not written; a sequence whose starts are not in order or exceed
 * rows or keys counts as empty.  out must not overlap q, k or v.  d_workspace
 * (16-byte aligned, NULL where it needs no bytes) holds nothing from one call to the
 * next; calls that may run at once need one each.  Asynchronous on `stream`, whose
 * device is current; no allocation; can be captured. */
SC_API sc_status prompt_attention(const sc_prompt* p, void* d_workspace, void* stream);

/* ---- a key/value cache in 4 bits ------------------------------------------------ */

#define SC_KV4_PAGE 64               /* tokens of a page */
#define SC_KV4_MAX_HEADS 1024
#define SC_KV4_MAX_SEQS 65536
#define SC_KV4_MAX_WIDTH (1 << 24)   /* pages of a sequence */
#define SC_KV4_MAX_ROWS 16
#define SC_KV4_MAX_GROUP 64

/* One layer's cache: pages of 64 tokens, each with the codes and scales of all
 * its heads' keys and values (the formats of 4-bit weights, groups along
 * head_dim), kv4_page_bytes per page and head.  Where inside a page a token's
 * codes lie follows the attention kernel's loads: pages are written by
 * kv4_append and read back by kv4_read.
 * Of a cache that evicts, every token has for each head its accumulated
 * attention weight and its position in the sequence. */
typedef struct {
  int32_t format;            /* SC_FP4_NV or SC_FP4_MX */
  int32_t head_dim;          /* 64, 128 or 256 */
  int32_t kv_heads;          /* <= SC_KV4_MAX_HEADS */
  int32_t n_pages;           /* > 0 */
  void* d_pages;             /* [n_pages][kv_heads][kv4_page_bytes], 16-byte aligned */
  float* d_weights;          /* [n_pages][kv_heads][64], 16-byte aligned, or NULL */
  int32_t* d_positions;      /* [n_pages][kv_heads][64], 16-byte aligned; NULL with d_weights */
  const float* d_k_scale;    /* NVFP4: one float > 0 that all keys' group scales are multiplied by; NULL stands for 1 */
  const float* d_v_scale;    /* the same for values */
} sc_kv4_cache;

/* Sequences of a batch: place p of sequence b is token p % 64 of page
 * d_table[b * ld_table + p / 64], for 0 <= p < d_lens[b].  d_lens counts the
 * tokens that come with the call.  A length below 0 or above 64 * width and a
 * page outside of the cache are found by the kernels: what each call says of it. */
typedef struct {
  int32_t n_seqs;            /* <= SC_KV4_MAX_SEQS */
  int32_t width;             /* entries of a table row, <= SC_KV4_MAX_WIDTH */
  int64_t ld_table;
  const int32_t* d_table;
  const int32_t* d_lens;     /* [n_seqs] */
} sc_kv4_seqs;

/* Keys and values of packed tokens: element d of token t and head h of k at t *
 * k_token + h * k_head + d, and so for v. */
typedef struct {
  int32_t type;              /* SC_DTYPE_F32, SC_DTYPE_BF16 or SC_DTYPE_F16 */
  void* d_k;
  void* d_v;
  int64_t k_token, k_head, v_token, v_head;
} sc_kv4_rows;

/* Bytes of one page of one head, keys and values. */
SC_API sc_status kv4_page_bytes(int32_t format, int32_t head_dim, size_t* bytes);

/* Quantises tokens into the cache: sequence b has the tokens d_starts[b] ..
 * d_starts[b+1]-1 (NULL: tokens / n_seqs each), which are its last: the last one
 * goes to place d_lens[b] - 1.  Codes and scales follow fp4_quantize with a given
 * scale.  A cache with weights gets weight 0 (kv4_attention with `accumulate` adds
 * to it; the last rows of a prompt, given to it before an eviction, give all of the
 * prompt's tokens weights) and the position d_positions[token]
 * (NULL: the place).  tokens * kv_heads * head_dim < 2^32, here and in kv4_read.
 * Tokens outside of the sequences, places that are not in the table and pages
 * outside of the cache are not written.  No two tokens of a call may have one place
 * of one page.  Asynchronous on `stream`, whose device is
 * current; no workspace, no allocation; can be captured. */
SC_API sc_status kv4_append(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, const sc_kv4_rows* rows, int32_t tokens,
                            const int32_t* d_starts, const int32_t* d_positions, void* stream);

/* Reads the last tokens of each sequence back, addressed as in kv4_append: code *
 * group scale * scale, rounded to fp32 once and then to rows->type.  Tokens
 * outside of the sequences are not written; places or pages that are not there
 * read as NaN. */
SC_API sc_status kv4_read(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, const sc_kv4_rows* rows, int32_t tokens,
                          const int32_t* d_starts, void* stream);

/* Queries of the last `rows` tokens of every sequence: element d of row r and
 * head h of sequence b at b * q_stride[0] + r * q_stride[1] + h * q_stride[2] +
 * d, and so for out. */
typedef struct {
  int32_t type;              /* of q and out: SC_DTYPE_BF16 or SC_DTYPE_F16 */
  int32_t rows;              /* 1 .. SC_KV4_MAX_ROWS: a token and its drafts */
  int32_t q_heads;           /* a multiple of kv_heads, up to SC_KV4_MAX_GROUP times */
  float scale;               /* > 0, <= SC_ATTENTION_MAX_SCALE */
  const void* d_q;
  void* d_out;
  int64_t q_stride[3], out_stride[3];
} sc_kv4_query;

/* Bytes of device workspace that kv4_attention needs. */
SC_API sc_status kv4_attention_workspace_bytes(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t rows,
                                               int32_t q_heads, int32_t accumulate, size_t* bytes);

/* Attention over the cache: row r of sequence b sees the places below d_lens[b]
 * - rows + r + 1 (its own token and those before it).  n_seqs * rows * q_heads <=
 * 2^23.  out = softmax(scale q k^T) v; a row that sees nothing gets 0.  With `accumulate` every token's weight
 * grows by the sum of its probabilities over the rows and over the query heads of
 * its head; sequences of such a call must not share pages.  Products are exact;
 * sums and softmax statistics are fp32 in a fixed order; P keeps 11 bits (NVFP4)
 * or 16 (MXFP4).  Rows of a sequence whose length cannot be are NaN, and so are
 * rows that see a page outside of the cache, or anything where the keys' scale is
 * NaN, infinite or negative (and the weights that those add to).
 * d_workspace (256-byte aligned) holds nothing from one call to the next; calls
 * that may run at once need one each.  out must not overlap q.  Asynchronous on
 * `stream`, whose device is current; no allocation; can be captured. */
SC_API sc_status kv4_attention(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, const sc_kv4_query* query,
                               int32_t accumulate, void* d_workspace, void* stream);

/* Bytes of device workspace that kv4_evict needs. */
SC_API sc_status kv4_evict_workspace_bytes(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t keep,
                                           size_t* bytes);

/* Cuts every sequence of more than `keep` tokens down to `keep`: of each head the
 * tokens at positions below `sinks` or among the last `recent` positions stay
 * before all others, then those with the largest weights (NaN largest), equal
 * ones by place.  recent + sinks <= keep.  Tokens that stay keep their places
 * below `keep`; those behind move, in order, into the places that became free,
 * with their weights and positions, so a sequence's tokens are not in order
 * afterwards (attention does not depend on it; later calls to kv4_append should
 * give positions).  d_new_lens[b] = min(d_lens[b], keep); a sequence with a
 * length or page that cannot be stays as it is and keeps its length.  Sequences
 * that are cut must not share pages.  n_seqs * kv_heads <= 2^17.  d_new_lens [n_seqs]
 * must not overlap d_lens.  d_workspace (4-byte aligned) holds nothing from one call
 * to the next; calls that may run at once need one each.
 * Asynchronous on `stream`, whose device is current; no allocation; can be
 * captured. */
SC_API sc_status kv4_evict(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t keep, int32_t recent,
                           int32_t sinks, int32_t* d_new_lens, void* d_workspace, void* stream);

/* Message for the last non-OK status returned on this thread. */
SC_API const char* slotcache_last_error(void);

/* Frees the pinned backing store and the handle (synchronizes the device).
 * The caller's device buffers are not freed. */
SC_API void slotcache_destroy(sc_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* SLOTCACHE_H */
