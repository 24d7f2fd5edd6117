/*
 * pagedattn -- batched ragged attention over a paged KV cache, for one
 * GB300 GPU (sm_103a).  Plain C ABI: plain pointers and sizes, no C++ or
 * framework types cross it.
 *
 * The problem statement follows the FlashInfer issue "How are prefill and
 * decode kernels different?" (the timing script and its
 * BatchDecodeWithPagedKVCacheWrapper / BatchPrefillWithPagedKVCacheWrapper
 * calls): a batch of requests, request b owning
 *
 *   - qo_len_b query rows packed in q[T, Hq, D] between qo_indptr[b] and
 *     qo_indptr[b+1] (prefill chunks have qo_len > 1, decodes qo_len = 1);
 *   - kv_len_b keys/values stored in the pages kv_page_indices[
 *     kv_page_indptr[b] .. kv_page_indptr[b+1]) of the cache
 *     kv_cache[num_pages, 2, page_size, Hkv, D] ("NHD": index 0 of the
 *     second dimension holds K, index 1 holds V); every page is full except
 *     the last, which holds kv_last_page_len[b] slots, 1 <= last <= page_size.
 *     kv_len_b = (pages_b - 1) * page_size + last_b.
 *
 * Query head h reads kv head h / (Hq / Hkv) (grouped-query attention).  Query
 * row i of request b sits at absolute position kv_len_b - qo_len_b + i and,
 * with causal = 1, sees keys [0, kv_len_b - qo_len_b + i] (the mask aligned
 * to the bottom-right, so new tokens appended after a shared prefix -- the
 * vLLM issue "Question about efficient memory sharing (prefix sharing)" --
 * see the whole prefix, and fully masked tails are never visited, as the
 * llama.cpp discussion "Pad for prefill stage?" describes).  With scale =
 * 1/sqrt(D):
 *
 *   out[row, h, :] = sum_t softmax_t(scale * q[row,h,:] . K[t,:]) * V[t,:]
 *   lse[row, h]    = ln sum_t exp(scale * q[row,h,:] . K[t,:])   (natural log)
 *
 * Several page tables may list the same physical page (prefix sharing): the
 * library only reads the cache.
 *
 * Life cycle (the script's begin_forward / forward / end_forward):
 *   pagedattn_plan()          once per batch: host work, one H2D copy
 *   pagedattn_run()           any number of times, asynchronous, no alloc
 *   pagedattn_plan_destroy()  when the batch is done
 *
 * Errors: every call returns a pagedattn_status; the text of the last error
 * on the calling thread is pagedattn_last_error().  No call aborts, prints or
 * throws.
 */
#ifndef PAGEDATTN_H_
#define PAGEDATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PAGEDATTN_API __attribute__((visibility("default")))
#else
#define PAGEDATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* CUDA stream handle, identical to cudaStream_t (a CUstream_st pointer). */
typedef struct CUstream_st* pagedattn_stream_t;

typedef struct pagedattn_plan_s* pagedattn_plan_t; /* opaque, owned by the library */

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,         /* malformed indptr / page ids / lengths / pointers  */
  PA_ERR_UNSUPPORTED = 2,         /* head_dim, page_size, dtype or group size not built */
  PA_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < pagedattn_workspace_size()       */
  PA_ERR_CUDA = 4,                /* a CUDA runtime call failed (message has the code)  */
  PA_ERR_DEVICE_CHECK = 5,        /* an in-kernel check fired (see device_status)       */
  PA_ERR_TIMEOUT = 6              /* an in-kernel wait gave up after its bound          */
} pagedattn_status;

typedef enum { PA_FP16 = 0, PA_BF16 = 1 } pagedattn_dtype;

/* Optional planner settings; pass NULL for the defaults (all zero). */
typedef struct {
  int32_t num_sms;             /* SMs to plan for; 0 = ask the current device        */
  int32_t force_prefill;       /* 1: every request uses the tcgen05 prefill kernel    */
  int32_t decode_chunk_pages;  /* > 0: pages per decode split (default: see plan)    */
  int32_t prefill_chunk_tiles; /* > 0: 128-key tiles per prefill split               */
  int32_t force_cp_async;      /* 1: stage K/V with cp.async instead of TMA           */
  int32_t decode_cuda_cores;   /* 1: single-token requests at group sizes <= 8 run on
                                  the CUDA-core decode kernel, and multi-token
                                  requests all go to the prefill kernel (default:
                                  the warp-MMA small-query kernel, see plan)        */
  int32_t kv_layout;           /* PA_LAYOUT_NHD (default) or PA_LAYOUT_HND: see below */
  int32_t prefill_q_tiles;     /* 128-row query tiles per prefill work item: 1 or 2;
                                  0 = the planner's choice (see plan).  head_dim 256
                                  takes 1 only                                      */
  int32_t wait_limit_cycles;   /* test hook: > 0 bounds every in-kernel pipeline wait
                                  at that many SM clock cycles instead of about 2 s,
                                  and makes one thread of every CTA first wait on a
                                  barrier that nothing completes, so the waits give
                                  up (the run then reports PA_DEV_TIMEOUT through
                                  device_status and leaves out / lse undefined);
                                  0 = the default                                   */
  int32_t reserved[1];         /* must be 0                                          */
} pagedattn_options;

/*
 * Cache layouts (pagedattn_options.kv_layout).  Both hold, per physical page,
 * the page_size K rows and then the page_size V rows of every kv head; the
 * FlashInfer timing script passes "NHD" and the alternative it implies keeps
 * each head's rows together:
 *   PA_LAYOUT_NHD  kv_cache[num_pages][2][page_size][num_kv_heads][head_dim]
 *   PA_LAYOUT_HND  kv_cache[num_pages][2][num_kv_heads][page_size][head_dim]
 * The results are identical (bit for bit) for the same logical cache.
 */
#define PA_LAYOUT_NHD 0
#define PA_LAYOUT_HND 1

/* Stage bits for pagedattn_run_stages. */
#define PA_STAGE_PREFILL 1u
#define PA_STAGE_DECODE 2u
#define PA_STAGE_MERGE 4u
#define PA_STAGE_ALL 7u

/* Status bits the kernels OR into the device status word. */
#define PA_DEV_TIMEOUT 1
#define PA_DEV_BAD_INDEX 2
#define PA_DEV_NO_PAGES 4 /* build_tables: the free stack holds too few pages            */
#define PA_DEV_NO_ROOM 8  /* build_tables: block_table_width, max_tokens or max_pages;
                             blocks: max_pages                                         */

/*
 * Build the work partition for one batch ("auxiliary data structures" that
 * begin_forward builds, in the timing script).
 *
 * qo_indptr        host, int32[batch_size + 1], [0] == 0, nondecreasing.
 * kv_page_indptr   host, int32[batch_size + 1], [0] == 0, nondecreasing.
 * kv_page_indices  host, int32[kv_page_indptr[batch_size]], each in [0, num_pages).
 * kv_last_page_len host, int32[batch_size], in [1, page_size] for every request
 *                  that has pages.
 * num_qo_heads, num_kv_heads: num_qo_heads a positive multiple of num_kv_heads;
 *                  the group size num_qo_heads / num_kv_heads must divide 128.
 * head_dim         64, 128 or 256 (at 256 decode runs on the CUDA-core kernel
 *                  for single-token requests at group size <= 8, everything
 *                  else on the tensor-core prefill kernel).  page_size: a
 *                  power of two in [1, 128].
 * causal           1: bottom-right causal mask (qo_len <= kv_len required);
 *                  0: every row sees all kv_len keys.
 * workspace        caller-owned device buffer (the wrapper's workspace in the
 *                  script); the plan writes its metadata (work items, page ids,
 *                  merge map) to its start with one cudaMemcpyAsync on `stream`
 *                  and keeps fp32 split-KV partial states after it.  The copy's
 *                  source is pageable host memory, so the call may hold the
 *                  host until `stream` reaches it: a serving loop that plans
 *                  the next step while the current one runs passes a stream
 *                  that is not queued behind the running kernels (its upload
 *                  stream).  It must stay
 *                  allocated and untouched while the plan is used.  NULL builds a
 *                  host-only plan (metadata inspection; run() then fails).
 * workspace_bytes  its size; PA_ERR_WORKSPACE_TOO_SMALL below the size
 *                  pagedattn_workspace_size() reports.
 * opts             NULL or settings (see pagedattn_options).
 * out_plan         receives the handle; destroy it with pagedattn_plan_destroy.
 *
 * Host arrays are read during the call only; the library keeps its own copy.
 * The call is synchronous on the host and asynchronous on the device (the
 * metadata copy is queued on `stream`).
 */
PAGEDATTN_API pagedattn_status pagedattn_plan(const int32_t* qo_indptr, const int32_t* kv_page_indptr,
                                const int32_t* kv_page_indices, const int32_t* kv_last_page_len,
                                int32_t batch_size, int32_t num_qo_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t page_size, int32_t num_pages,
                                pagedattn_dtype dtype, int32_t causal, void* workspace,
                                size_t workspace_bytes, const pagedattn_options* opts,
                                pagedattn_stream_t stream, pagedattn_plan_t* out_plan);

/*
 * Bytes of workspace the same arguments need (metadata + partial states).
 * Pure host computation; writes *bytes.
 */
PAGEDATTN_API pagedattn_status pagedattn_workspace_size(const int32_t* qo_indptr, const int32_t* kv_page_indptr,
                                          const int32_t* kv_page_indices,
                                          const int32_t* kv_last_page_len, int32_t batch_size,
                                          int32_t num_qo_heads, int32_t num_kv_heads,
                                          int32_t head_dim, int32_t page_size, int32_t num_pages,
                                          pagedattn_dtype dtype, int32_t causal,
                                          const pagedattn_options* opts, size_t* bytes);

/*
 * Shared-prefix cascade (the vLLM issue "Question about efficient memory
 * sharing (prefix sharing)": requests that start from one system prompt
 * should share its attention work, not only its pages).
 *
 * The requests of group g -- consecutive in the batch: requests
 * [group_indptr[g], group_indptr[g+1]) -- all begin with the same prefix
 * of full pages prefix_page_indices[prefix_page_indptr[g] ..
 * prefix_page_indptr[g+1]), followed by their own pages as described by
 * kv_page_indptr / kv_page_indices / kv_last_page_len (which then count only
 * the keys after the prefix).  Request b of the group attends to
 * prefix_len_g + kv_len_b keys: exactly what pagedattn_plan computes for the
 * flattened page table (prefix pages, then the request's own), with the
 * bottom-right causal mask over the whole sequence.  Its query rows must lie
 * after the prefix (qo_len_b <= kv_len_b, the usual check on the request's
 * own keys), so each of them sees the whole prefix.
 *
 * The plan computes the prefix attention once for all query tokens of the
 * group (they are consecutive in q) as one unmasked prefill, the rest per
 * request, and merges the two with the split-KV merge; results agree with
 * the flattened plan within the usual tolerance (sums in another order).
 * A group with no prefix pages is planned like ordinary requests.
 */
typedef struct {
  const int32_t* group_indptr;        /* host, [num_groups + 1], [0] == 0, nondecreasing,
                                         [num_groups] == batch_size                       */
  const int32_t* prefix_page_indptr;  /* host, [num_groups + 1], [0] == 0, nondecreasing    */
  const int32_t* prefix_page_indices; /* host, the groups' full prefix pages, each in
                                         [0, num_pages)                                    */
  int32_t num_groups;                 /* >= 0; 0 plans like pagedattn_plan                 */
} pagedattn_prefix_groups;

/* pagedattn_plan with shared-prefix groups (NULL groups: pagedattn_plan). */
PAGEDATTN_API pagedattn_status pagedattn_plan_cascade(const pagedattn_prefix_groups* groups,
                                        const int32_t* qo_indptr, const int32_t* kv_page_indptr,
                                        const int32_t* kv_page_indices, const int32_t* kv_last_page_len,
                                        int32_t batch_size, int32_t num_qo_heads, int32_t num_kv_heads,
                                        int32_t head_dim, int32_t page_size, int32_t num_pages,
                                        pagedattn_dtype dtype, int32_t causal, void* workspace,
                                        size_t workspace_bytes, const pagedattn_options* opts,
                                        pagedattn_stream_t stream, pagedattn_plan_t* out_plan);

/* pagedattn_workspace_size for pagedattn_plan_cascade. */
PAGEDATTN_API pagedattn_status pagedattn_workspace_size_cascade(const pagedattn_prefix_groups* groups,
                                          const int32_t* qo_indptr, const int32_t* kv_page_indptr,
                                          const int32_t* kv_page_indices,
                                          const int32_t* kv_last_page_len, int32_t batch_size,
                                          int32_t num_qo_heads, int32_t num_kv_heads,
                                          int32_t head_dim, int32_t page_size, int32_t num_pages,
                                          pagedattn_dtype dtype, int32_t causal,
                                          const pagedattn_options* opts, size_t* bytes);

/*
 * Attention for the planned batch (the script's forward(q, kv_cache)).
 *
 * q        device, dtype[T, Hq, D] contiguous, 16-byte aligned (T = qo_indptr[B]).
 * kv_cache device, dtype[num_pages, 2, page_size, Hkv, D] contiguous, 16-byte aligned.
 * out      device, dtype[T, Hq, D], caller-allocated; every row of a request
 *          with qo_len >= 1 is written.
 * lse      device, float[T, Hq] natural-log sums, or NULL to skip.
 * stream   the stream every kernel is queued on.
 *
 * Launches the prefill kernel (tcgen05 / TMEM), the small-query kernels
 * (decode and requests of qo_len * G <= 32 rows: warp-level MMA, one launch
 * per row class, or the CUDA-core decode kernel) and, when some request was
 * split, the merge kernel, in that order on `stream`.  Allocates nothing and does not synchronise the host.
 * The kernels are launched with programmatic stream serialization: each may
 * begin its set-up while the kernel before it on `stream` finishes, and
 * waits for that kernel's completion before it reads q, kv_cache or partial
 * states or writes anything, so stream order holds for every buffer.  In-kernel
 * waits are bounded; a wait that gives up sets PA_DEV_TIMEOUT in the device
 * status word (read it with pagedattn_device_status).  Calls that overlap on
 * the device must use different workspaces (the partial states live there),
 * so two such calls need two plans.  Host threads may call run on one plan
 * at once: the plan's host-side state (its cache of TMA descriptors) is
 * locked; kernel launch settings are applied per device.
 */
PAGEDATTN_API pagedattn_status pagedattn_run(pagedattn_plan_t plan, const void* q, const void* kv_cache,
                               void* out, float* lse, pagedattn_stream_t stream);

/*
 * Same as pagedattn_run restricted to the stages in `stage_mask`
 * (PA_STAGE_* bits).  Running PREFILL, DECODE and MERGE in that order is
 * exactly pagedattn_run; used to time the kernels one by one.
 */
PAGEDATTN_API pagedattn_status pagedattn_run_stages(pagedattn_plan_t plan, const void* q, const void* kv_cache,
                                      void* out, float* lse, pagedattn_stream_t stream,
                                      uint32_t stage_mask);

/* Release a plan (end_forward in the script).  NULL is a no-op. */
PAGEDATTN_API pagedattn_status pagedattn_plan_destroy(pagedattn_plan_t plan);

/* Thread-local text of the last error ("" when none).  Never NULL. */
PAGEDATTN_API const char* pagedattn_last_error(void);

/*
 * Wait for `stream`, read the device status word of the plan's workspace
 * (PA_DEV_* bits OR-ed by the kernels since the plan or the last read) into
 * *flags and clear it.  Returns PA_ERR_TIMEOUT / PA_ERR_DEVICE_CHECK when a
 * bit is set, PA_OK otherwise.
 */
PAGEDATTN_API pagedattn_status pagedattn_device_status(pagedattn_plan_t plan, pagedattn_stream_t stream,
                                         int32_t* flags);

/*
 * Copy the plan metadata (exactly the bytes copied to the workspace) into
 * host_buf.  With host_buf NULL, only writes the size to *bytes; otherwise
 * *bytes is the buffer size on input and the bytes written on output.
 * Layout: int32 words, documented with the planner rules in the source.
 */
PAGEDATTN_API pagedattn_status pagedattn_debug_plan_dump(pagedattn_plan_t plan, void* host_buf, size_t* bytes);

/*
 * Test hook for the page-table walk: a kernel that resolves every logical
 * token t < kv_len_b of every request b (in request order) with the same
 * device index code the attention kernels use, writing the physical page id
 * and slot to page_out / slot_out (device, int32[sum_b kv_len_b]).
 * Asynchronous on `stream`.
 */
PAGEDATTN_API pagedattn_status pagedattn_debug_gather(pagedattn_plan_t plan, int32_t* page_out,
                                        int32_t* slot_out, pagedattn_stream_t stream);

/*
 * Decode without a device workspace.  The source pages have no counterpart
 * to this call; it exists for callers that cannot allocate device memory --
 * serving processes that reserve all free GPU memory for their KV cache up
 * front, and latency-critical code that must not call cudaFree (which
 * synchronises the device).
 *
 * Runs the decode kernel and the split merge of `plan` (build it with
 * pagedattn_plan and workspace = NULL) with the plan's metadata and split-KV
 * partial states in a fixed 16 MiB device array inside the library instead
 * of a caller workspace.  The array exists once per GPU that loads the
 * library and stays allocated until the process exits.  q, kv_cache, out and
 * lse are as for pagedattn_run.
 *
 * The batch must have no prefill items (every request has qo_len 0 or
 * qo_len * G <= 32 with the group size G = num_qo_heads / num_kv_heads in
 * {1, 2, 4, 8, 16}, and force_prefill is off; with decode_cuda_cores or at
 * head_dim 256, qo_len <= 1 and G <= 8): PA_ERR_UNSUPPORTED otherwise.  A plan whose metadata and partial
 * states exceed 16 MiB returns PA_ERR_WORKSPACE_TOO_SMALL (plan with a larger
 * decode_chunk_pages).  The call allocates no memory.  Its first call on a
 * device looks up the array's device address (cudaGetSymbolAddress) while
 * that device is current; make that first call before any stream capture.
 * Every call overwrites the array, whose contents are whatever the last call
 * left (the plan's metadata copy clears the in-kernel status word): calls
 * that overlap on the GPU -- on different streams or from different host
 * threads -- race and must not be issued.  The in-kernel status word of the
 * last call is read with pagedattn_noalloc_device_status.
 */
PAGEDATTN_API pagedattn_status pagedattn_run_decode_noalloc(pagedattn_plan_t plan, const void* q,
                                                            const void* kv_cache, void* out, float* lse,
                                                            pagedattn_stream_t stream);

/*
 * The device status word (PA_DEV_* bits) that the kernels of the last
 * pagedattn_run_decode_noalloc call on the current device left in the
 * library's no-alloc array: waits for `stream` (pass the stream of that
 * call), copies the word into *flags and returns PA_ERR_TIMEOUT /
 * PA_ERR_DEVICE_CHECK when a bit is set, PA_OK otherwise.  Allocates
 * nothing; the next no-alloc call clears the word.
 */
PAGEDATTN_API pagedattn_status pagedattn_noalloc_device_status(pagedattn_stream_t stream, int32_t* flags);

/* ------------------------------------------------------------------------
 * A decode step without the host: page tables built on the device, a cache
 * held in 4 bits, and attention over it.
 *
 * The entries below keep every length on the device, so that a whole step
 * (tables, append, attention) can be captured into one CUDA graph and
 * replayed while the requests grow.  All are asynchronous on `stream`,
 * allocate nothing and keep nothing between calls but what is documented;
 * pointers belong to the current device.  Two calls may overlap on the
 * device unless one writes what the other uses (outputs, cache rows, or the
 * workspace of pagedattn_kv4_run).
 *
 * Kernels OR PA_DEV_* bits into a status word in device memory that the
 * caller zeroes once and reads with pagedattn_status_word.
 */

/* Inputs of pagedattn_build_tables.  All arrays are device memory. */
typedef struct {
  const int32_t* qo_lens;     /* [batch_size] tokens that each request appends, >= 0     */
  const int32_t* kv_lens;     /* [batch_size] tokens that it has cached already, >= 0    */
  int32_t* block_table;       /* [batch_size][block_table_width] page ids, row b's first
                                 ceil(kv_lens[b] / page_size) held already; this step's
                                 new pages are entered behind them                       */
  const int32_t* free_pages;  /* [free_capacity] a stack of free page ids: the first
                                 *free_count are free and the top is the last of them    */
  const int32_t* free_count;  /* [1]                                                     */
  int64_t block_table_stride; /* entries between rows, >= block_table_width              */
  int32_t block_table_width, free_capacity, batch_size;
  int32_t page_size;          /* a power of two in [1, 128]                              */
  int32_t num_pages;          /* page ids lie in [0, num_pages)                          */
} pagedattn_tables_in;

/* Outputs of pagedattn_build_tables.  All arrays are device memory. */
typedef struct {
  int32_t* qo_indptr;        /* [batch_size + 1] exclusive sums of qo_lens               */
  int32_t* kv_page_indptr;   /* [batch_size + 1] exclusive sums of the pages, new ones
                                included                                                 */
  int32_t* new_page_indptr;  /* [batch_size + 1] exclusive sums of the pages taken       */
  int32_t* kv_page_indices;  /* [max_pages] the requests' pages one after the other;
                                entries from kv_page_indptr[batch_size] on are left      */
  int32_t* kv_last_page_len; /* [batch_size] slots of the last page, 0 without pages     */
  int32_t* kv_lens;          /* [batch_size] kv_lens + qo_lens; may be the input array   */
  int64_t* slot_mapping;     /* [max_tokens] page * page_size + slot of each new token,
                                request after request; -1 from qo_indptr[batch_size] on  */
  int32_t* positions;        /* [max_tokens] its position in its request; 0 from there on */
  int32_t* free_count;       /* [1] pages left on the stack; may be the input array      */
  int32_t* status;           /* [2] status word, and a word that builds count their
                                blocks in: zero both once                                */
  int32_t max_tokens, max_pages;
} pagedattn_tables_out;

/*
 * The tables of one step from its requests' lengths.  Request b needs
 * ceil((kv_lens[b] + qo_lens[b]) / page_size) pages; those it lacks come off
 * the top of the free stack in request order (the n-th page taken by the
 * whole batch is free_pages[*free_count - 1 - n]).  Requests of no tokens
 * and no pages are allowed.  The outputs are what pagedattn_plan takes (after
 * a copy to the host) and what pagedattn_kv4_append and pagedattn_kv4_run
 * read in place.
 *
 * All or nothing: where a length is negative or their sum passes
 * 2^31 - 1 - page_size (PA_DEV_BAD_INDEX), the stack is short (PA_DEV_NO_PAGES), or a row of the
 * block table, max_tokens or max_pages is (PA_DEV_NO_ROOM), the outputs are
 * those of an empty batch (indptr all 0, slot_mapping all -1, kv_lens and
 * free_count as they were) and the block table is left alone.  A page id
 * outside [0, num_pages) raises PA_DEV_BAD_INDEX and its tokens get slot -1.
 */
PAGEDATTN_API pagedattn_status pagedattn_build_tables(const pagedattn_tables_in* in, const pagedattn_tables_out* out,
                                        pagedattn_stream_t stream);

/*
 * A paged cache of 4-bit keys and values: e2m1 codes, two to a byte (the even
 * element of head_dim in the low four bits), and an e4m3 scale for each 16
 * elements along head_dim.  A value is code * scale * k_scale (or v_scale).
 *   NHD  codes [num_pages][2][page_size][num_kv_heads][head_dim / 2]
 *        scales[num_pages][2][page_size][num_kv_heads][head_dim / 16]
 *   HND  the same with page_size and num_kv_heads exchanged
 * Both device memory, 32-byte aligned.  Memory of slots that were never
 * written may hold anything.
 */
typedef struct {
  void* codes;
  void* scales;
  int32_t num_pages, page_size, num_kv_heads;
  int32_t head_dim;  /* 64, 128 or 256                       */
  int32_t kv_layout; /* PA_LAYOUT_NHD or PA_LAYOUT_HND       */
  float k_scale, v_scale;  /* in [1e-15, 1e15]               */
} pagedattn_kv4_cache;

/* Rows for pagedattn_kv4_append. */
typedef struct {
  const void* k;               /* device, dtype[num_tokens][num_kv_heads][head_dim], tokens
                                  k_stride elements apart (slices of a fused projection's
                                  output), 16-byte aligned                                  */
  const void* v;
  int64_t k_stride, v_stride;  /* multiples of 8                                            */
  void* k_values;              /* NULL, or device, dtype[num_tokens][num_kv_heads][head_dim]
                                  contiguous: the rows as later reads see them             */
  void* v_values;
  const int64_t* slot_mapping; /* device, [num_tokens] page * page_size + slot; a row with a
                                  negative slot is skipped                                  */
  int32_t* status;             /* device, status word                                       */
  int32_t num_tokens;
  pagedattn_dtype dtype;
} pagedattn_kv4_rows;

/*
 * Quantise rows into the cache.  Per block of 16 elements, with g the cache's
 * scale of K or V, each step rounded to nearest even: scale = e4m3(amax / (6 g)),
 * at most 448; code = e2m1(x / (scale * g)), beyond 6 to 6, and 0 where the
 * scale is 0.  A block with a NaN reads back as NaN; an infinity becomes the
 * block's largest value.  Slots at num_pages * page_size or beyond are skipped
 * and raise PA_DEV_BAD_INDEX.  The non-negative slots of one call must be
 * distinct: two rows for one slot may leave a mixture of both there.
 */
PAGEDATTN_API pagedattn_status pagedattn_kv4_append(const pagedattn_kv4_cache* cache, const pagedattn_kv4_rows* rows,
                                      pagedattn_stream_t stream);

/* The batch that pagedattn_kv4_run attends for.  Arrays are device memory. */
typedef struct {
  const int32_t* qo_indptr;        /* [batch_size + 1]                                    */
  const int32_t* kv_page_indptr;   /* [batch_size + 1]                                    */
  const int32_t* kv_page_indices;  /* [num_page_indices]                                  */
  const int32_t* kv_last_page_len; /* [batch_size]                                        */
  int32_t batch_size;
  int32_t num_page_indices;        /* entries of kv_page_indices; also the host's only bound of
                                      the batch's keys, by which the kernels are chosen: with
                                      one far larger than the pages in use the results are as
                                      exact, but short prompts take up to half as long again */
  int32_t num_tokens;              /* rows of q, out and lse, >= qo_indptr[batch_size]    */
  int32_t max_qo_len;              /* bound of the requests' query lengths: chooses the
                                      kernels (a longer request is computed too, slower;
                                      see the note on NaN below)                          */
  int32_t num_qo_heads, causal;
  pagedattn_dtype dtype;           /* of q and out                                        */
} pagedattn_kv4_batch;

/* Bytes of workspace that pagedattn_kv4_run needs on the current device. */
PAGEDATTN_API pagedattn_status pagedattn_kv4_workspace_size(int32_t num_qo_heads, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t max_qo_len, size_t* bytes);

/*
 * Attention as pagedattn_run computes it (see the top of this file), over a
 * 4-bit cache and with the batch's tables in device memory.  Any group size
 * num_qo_heads / num_kv_heads up to 128; any lengths.  A row that sees no key
 * (kv_len 0, or causal with qo_len > kv_len) gets zeros and lse = -inf.  A NaN
 * of K or V reaches the rows that see its key and no others, except that with
 * max_qo_len <= 1 the rows of a longer request may share their NaN.  Logits
 * have to stay within fp32's range; values of a bf16 row of q are off by at most
 * 2^-38 of the row's largest.  Rows of q from qo_indptr[batch_size] on are not
 * read, and rows of out and lse not written.
 *
 * q         device, dtype[num_tokens][num_qo_heads][head_dim], tokens q_stride
 *           elements apart (a multiple of 8), 16-byte aligned.
 * out       device, dtype[num_tokens][num_qo_heads][head_dim], 16-byte aligned; must not
 *           overlap q.
 * lse       device, float[num_tokens][num_qo_heads], or NULL.
 * workspace device, 256-byte aligned, pagedattn_kv4_workspace_size() bytes: zero
 *           it once, before its first run.  Its first word is the status word.
 *           Calls that overlap on the device need different workspaces; runs of
 *           other shapes or batches may share one, one after the other.
 *
 * A table entry that cannot be (indptr out of order or out of range, a last
 * page length outside [1, page_size]) leaves its request's rows unwritten, a
 * page id outside [0, num_pages) is read as page 0; both raise
 * PA_DEV_BAD_INDEX.
 */
PAGEDATTN_API pagedattn_status pagedattn_kv4_run(const pagedattn_kv4_cache* cache, const pagedattn_kv4_batch* batch,
                                   const void* q, int64_t q_stride, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, pagedattn_stream_t stream);

/* ------------------------------------------------------------------------
 * A step over the 16-bit cache without the host: rotary positions, rows
 * appended with the rotation on the way, bounds of each page's keys, the
 * pages that a query attends to, and the attention over them.  As for the
 * entries above: asynchronous on `stream`, nothing allocated or kept, tables
 * in device memory, PA_DEV_* bits in a status word, and two calls may overlap
 * on the device unless one writes what the other uses.
 */

/*
 * A rotation by position.  The first rotary_dim values of a head are pairs:
 * value i and value i + rotary_dim / 2, or with `interleaved` values 2 i and
 * 2 i + 1.  Pair i = (a, b) at position x becomes
 *   (a cos - b sin, b cos + a sin) * scale,  angle = 2 pi * x * turns[i] / 2^64
 * in fp32, rounded once; values behind the pairs stay as they are.  turns[i] is
 * the pair's turns a position modulo 1, as a 64-bit fraction: the product modulo 2^64 is
 * exact, and its cosine is taken of the fraction in fp32, off by less than 2^-25 turns at any
 * position.
 */
typedef struct {
  const uint64_t* turns; /* device, [rotary_dim / 2], 8-byte aligned                             */
  const int32_t* axes;   /* device, [rotary_dim / 2]: the axis whose position turns the pair, in
                            [0, num_axes) (others count as 0); or NULL, axis 0 for all          */
  int32_t num_axes;      /* positions a token: 1, or one for each of time, height, width ...    */
  int32_t rotary_dim;    /* a multiple of 16, at most head_dim                                  */
  int32_t interleaved;
  float scale;
} pagedattn_rotation;

/* Rows for pagedattn_rope.  Tokens are strides elements apart (multiples of 8). */
typedef struct {
  const void* q; /* device, dtype[num_tokens][num_q_heads][head_dim], 16-byte aligned            */
  const void* k; /* likewise with num_k_heads, or NULL with num_k_heads 0                        */
  void* q_out;   /* may be q (with its stride), otherwise must not overlap it; likewise k_out    */
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  const int32_t* positions; /* device, [num_axes][num_tokens], axes position_stride entries apart
                               (0: one row for all axes)                                      */
  int64_t position_stride;
  int32_t num_tokens, num_q_heads, num_k_heads;
  int32_t head_dim; /* a multiple of 16, at most 256                                             */
  int32_t inverse;  /* rotate by the negative angle: the gradient of the rotation (and, with scale
                       1, the rotation back)                                               */
  pagedattn_dtype dtype;
} pagedattn_rope_rows;

/* Rotate the rows of q and k by their positions. */
PAGEDATTN_API pagedattn_status pagedattn_rope(const pagedattn_rotation* rotation, const pagedattn_rope_rows* rows,
                                pagedattn_stream_t stream);

/*
 * A paged cache of 16-bit keys and values, laid out as pagedattn_run reads it,
 * with the bounds of its keys where pages are to be selected:
 *   bounds        [num_pages][num_kv_heads][2][head_dim] codes of the largest (0) and
 *                 the smallest (1) value of each channel over the page's keys
 *   bound_scales  [num_pages][num_kv_heads] what code 1 stands for
 * With a the largest magnitude over the page's keys and channels, and f = 127 * (1 / a):
 * the scale is a * (1 / 127) and the codes min(127, ceil(x * f)) of the largest x and
 * max(-127, floor(x * f)) of the smallest, each step rounded to fp32: but for these
 * roundings they enclose the keys (127 * scale may lie 2^-23 of it below a).  (a below 2^-100 counts as 0: scale and codes 0.  Where a
 * key is NaN or infinite the scale is infinite and the codes 127 and -127.)
 */
typedef struct {
  void* data;          /* device, 16-byte aligned                                  */
  int8_t* bounds;      /* device, 16-byte aligned, or NULL: no bounds are kept     */
  float* bound_scales; /* device, or NULL with bounds                              */
  int32_t num_pages, page_size, num_kv_heads;
  int32_t head_dim;    /* 64, 128 or 256                                           */
  int32_t kv_layout;   /* PA_LAYOUT_NHD or PA_LAYOUT_HND                           */
  pagedattn_dtype dtype;
} pagedattn_kv_cache;

/* Rows for pagedattn_kv_append.  Tokens are strides elements apart (multiples of 8). */
typedef struct {
  const void* k; /* device, dtype[num_tokens][num_kv_heads][head_dim], 16-byte aligned          */
  const void* v;
  const void* q; /* device, dtype[num_tokens][num_qo_heads][head_dim] to be rotated too, or NULL */
  void* q_out;   /* may be q (with its stride), otherwise must not overlap it                    */
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  const int64_t* slot_mapping; /* device, [num_tokens] page * page_size + slot; a row with a
                                  negative slot is skipped (its q is rotated all the same)      */
  const int32_t* positions;    /* device, [num_axes][num_tokens]; not used without a rotation    */
  int64_t position_stride;
  int32_t* status;             /* device, status word                                           */
  int32_t num_tokens, num_qo_heads;
} pagedattn_kv_rows;

/*
 * Append rows to the cache: k rotated where a rotation is given (NULL: as it
 * is), v as it is; and q rotated into q_out.  Slots at num_pages * page_size or
 * beyond are skipped and raise PA_DEV_BAD_INDEX.  The non-negative slots of
 * one call must be distinct: two rows for one slot may leave a mixture of both
 * there.  Where the cache has bounds, those of the pages written to are made
 * anew, as by pagedattn_kv_bounds, whose order of the slots is then asked for here too
 * (rows in any other order: a cache without bounds over the same data, then
 * pagedattn_kv_bounds with the slots sorted).
 */
PAGEDATTN_API pagedattn_status pagedattn_kv_append(const pagedattn_kv_cache* cache, const pagedattn_rotation* rotation,
                                     const pagedattn_kv_rows* rows, pagedattn_stream_t stream);

/*
 * The bounds of the pages that the slots name, each over its slots from 0 to
 * the one named last.  The slots of one page have to stand together in
 * ascending order, as pagedattn_build_tables lays them out: none of another page
 * between them.  Negative ones may stand anywhere and are skipped; those beyond the
 * cache too, which raises PA_DEV_BAD_INDEX, as does a slot behind a larger one or itself of
 * its page.  (Of a page whose slots stand apart, with another page's between them, the bounds
 * may be those of its keys up to any of the slots' groups.)
 */
PAGEDATTN_API pagedattn_status pagedattn_kv_bounds(const pagedattn_kv_cache* cache, const int64_t* slot_mapping,
                                     int32_t num_tokens, int32_t* status, pagedattn_stream_t stream);

/* The batch of pagedattn_select_blocks and pagedattn_blocks_run; a block is a page's worth of
 * a request's keys, counted from 0.  Arrays are device memory. */
typedef struct {
  const int32_t* qo_indptr;        /* [batch_size + 1]                                    */
  const int32_t* kv_page_indptr;   /* [batch_size + 1]                                    */
  const int32_t* kv_page_indices;  /* [num_page_indices]                                  */
  const int32_t* kv_last_page_len; /* [batch_size]                                        */
  int32_t batch_size, num_page_indices;
  int32_t num_tokens;              /* rows of q, blocks, out and lse, >= qo_indptr[batch_size] */
  int32_t num_qo_heads;
  int32_t num_blocks;              /* entries of a list, in [1, 4096]                     */
  int32_t first, last;             /* blocks that are always selected: the first ones, and the
                                      last ones up to the query's own; first >= 0, last >= 1,
                                      first + last <= num_blocks                          */
  int32_t max_pages;               /* most pages of a request                             */
  int32_t max_qo_len;              /* bound of the requests' query lengths, by which the kernels
                                      are chosen (a longer request is computed too, slower) */
} pagedattn_block_batch;

/* Bytes of workspace that the two calls below need on the current device, by the batch's sizes alone. */
PAGEDATTN_API pagedattn_status pagedattn_blocks_workspace_size(int32_t num_kv_heads, int32_t head_dim,
                                                 int32_t page_size, const pagedattn_block_batch* batch,
                                                 size_t* bytes);

/*
 * The blocks that each query attends to: for token t and kv head h the list
 * blocks[t][h][num_blocks], ascending, -1 behind its end.  A query at position x
 * (aligned as in pagedattn_run with causal = 1) has the blocks 0 .. x / page_size.
 * With no more than num_blocks of them all are listed; otherwise the first and
 * the last ones, and of the others those of the largest scores, of equal ones the
 * lowest.  The score bounds the sum over the group's query heads of q . key
 * for every key of the block from above, up to the rounding of q:
 *   x = rint(q * 2^e) for the group's heads, e such that their largest magnitude
 *       lies in [2^14, 2^15); u, l = the sums over the heads of max(x, 0) and min(x, 0)
 *   codes c = rint((u, l) * (127 * (1 / max(|u|, |l|))))      (each step in fp32; 0 where all are 0)
 *   score = scale of the block * sum over channels of (c_u * largest + c_l * smallest)
 * The sums are of whole numbers, so a score has the same bits in any batch.  (Requests of many
 * tokens are scored in tiles of 16 tokens where max_pages is at most 8192, else token by token.)
 * A NaN of the product (0 times an infinite scale) counts as infinity; a group
 * with a NaN or infinity in q has codes of 0.
 *
 * Rows of queries that have more than max_pages blocks get -1 throughout, and
 * PA_DEV_NO_ROOM is raised; table entries that cannot be leave their rows
 * unwritten, a page id outside [0, num_pages) is read as page 0, and both raise
 * PA_DEV_BAD_INDEX.  Rows from qo_indptr[batch_size] on are not written.
 *
 * q         device, the cache's dtype[num_tokens][num_qo_heads][head_dim], tokens q_stride
 *           elements apart (a multiple of 8), 16-byte aligned.
 * workspace device, 256-byte aligned, pagedattn_blocks_workspace_size() bytes: zero it once.
 *           Its first word is the status word.  Calls that overlap on the device need
 *           different workspaces; one after the other they may share one, of any sizes of
 *           this call and the next, but not with pagedattn_kv4_run.
 */
PAGEDATTN_API pagedattn_status pagedattn_select_blocks(const pagedattn_kv_cache* cache, const pagedattn_block_batch* batch,
                                         const void* q, int64_t q_stride, int32_t* blocks, void* workspace,
                                         size_t workspace_bytes, pagedattn_stream_t stream);

/*
 * Attention of each query over the keys of its listed blocks up to its own
 * position; softmax, out and lse as for pagedattn_run.  The lists are those of
 * pagedattn_select_blocks or the caller's own: ascending, negative entries behind
 * them; blocks behind the query's own are skipped.  A query that sees no key gets
 * zeros and lse = -inf.  So does one whose list is not ascending or names a
 * block twice (PA_DEV_BAD_INDEX is raised), or who has more than max_pages blocks
 * (PA_DEV_NO_ROOM).  Entries beyond the request's pages are skipped and raise
 * PA_DEV_BAD_INDEX, as do tables and page ids as above.  Rows from
 * qo_indptr[batch_size] on are neither read nor written.  out must not overlap q.
 *
 * Requests of few tokens (up to 32 packed rows) read the keys of each token by
 * itself.  Longer ones read those of many tokens together, where max_qo_len allows for them, pages have 8 slots or more and max_pages is at most 51200 /
 * (1 + W), with W the number of 32s, rounded up, in 256 / (heads of a group) tokens (half as many at
 * head_dim 256).  There a NaN or an infinity of K or V may reach other tokens of its request and
 * kv head, weights are rounded to the values' type (of bf16 values by up to 2^-8) but for
 * tokens of fewer than 128 keys, and logits have to stay below 2^26 in magnitude.
 */
PAGEDATTN_API pagedattn_status pagedattn_blocks_run(const pagedattn_kv_cache* cache, const pagedattn_block_batch* batch,
                                      const int32_t* blocks, const void* q, int64_t q_stride, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, pagedattn_stream_t stream);

/*
 * Wait for `stream`, read the status word *word (device memory) into *flags
 * and clear it.  Returns PA_ERR_TIMEOUT / PA_ERR_DEVICE_CHECK when a bit is
 * set, PA_OK otherwise.
 */
PAGEDATTN_API pagedattn_status pagedattn_status_word(int32_t* word, pagedattn_stream_t stream, int32_t* flags);

/* Library version as "major.minor.patch". */
PAGEDATTN_API const char* pagedattn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H_ */
