/*
 * il.h -- C ABI of the shared-input batched linear for GB300 (sm_103a).
 *
 * One call runs several matmul jobs over one shared fp32 activation:
 *     y_j[t][n_out_j] = x[t][n_in] * W_j^T        (W_j stored [n_out_j][n_in])
 * following the accelerator backend contract of oxinfer 0.0.0, src/gpu.rs:
 * struct `Job` (one matmul of a batch sharing x), `Backend::upload` (prepare
 * device state for one weight) and `Backend::matmul` (all jobs of a batch in
 * one submission).  There is no CPU fallback: an error returns a negative
 * status and launches nothing.
 *
 * Weight storage formats (enum `WeightRef` of the same page; the page names
 * Q8 and Q4 without defining them, this library fixes them as follows):
 *   IL_BF16: u16 bit patterns of bf16, host layout u16 w[n_out][n_in].
 *   IL_Q8  : symmetric int8, one fp32 scale per 32-element block along n_in;
 *            host layout i8 q[n_out][n_in], then f32 d[n_out][n_in/32]
 *            starting at byte n_out*n_in.  w = fp32(d*q).
 *   IL_Q4  : symmetric signed 4-bit (two's complement), two per byte, element
 *            2k in bits 0-3 of byte k and 2k+1 in bits 4-7; one fp32 scale
 *            per 32-block; host layout u8 p[n_out][n_in/2], then
 *            f32 d[n_out][n_in/32] starting at byte n_out*n_in/2.
 *
 * Threading: every entry point is thread-safe.  The library works on the
 * CUDA device that is current on the calling thread.  What it keeps per
 * stream it keeps per thread too for cudaStreamPerThread, one handle for a
 * stream of each thread.
 */
#ifndef IL_H_
#define IL_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define IL_VERSION 3

/* Storage format of a weight (oxinfer src/gpu.rs, enum WeightRef: the first three) or of a
 * K/V cache (IL_BF16, IL_Q8 and IL_A4, which il_kv describes). */
typedef enum { IL_BF16 = 0, IL_Q8 = 1, IL_Q4 = 2, IL_A4 = 3 } il_format;

/* Status codes.  IL_OK is 0; every error is negative.  An entry point that
 * returns an error has launched no work and written no output. */
typedef enum {
  IL_OK = 0,
  IL_ERR_ARG = -1,            /* null pointer, negative size, misaligned or overlapping buffer */
  IL_ERR_SHAPE = -2,          /* n_in / n_out inconsistent with a handle, or not a legal size */
  IL_ERR_FORMAT = -3,         /* unknown storage format */
  IL_ERR_HANDLE = -4,         /* freed, forged or other-device weight handle */
  IL_ERR_OOM = -5,            /* device allocation failed */
  IL_ERR_CUDA = -6,           /* CUDA runtime or launch error */
  IL_ERR_DEVICE_TIMEOUT = -7, /* a device-side wait gave up (see il_check_device_status) */
  IL_ERR_UNSUPPORTED = -8     /* no sm_103a device current, or a size beyond a documented limit */
} il_status;

/* Opaque device weight (the page's `DeviceWeight`).  Owned by the caller,
 * released with il_free_weight. */
typedef struct il_weight il_weight;

/* One job of a batch (the page's `Job`): y[t][n_out] = x[t][n_in] * W^T.
 *   w     : handle from il_upload_weight; its n_in must equal the batch n_in.
 *   n_out : must equal the handle's n_out.
 *   y     : DEVICE pointer (HOST pointer for il_matmul_batch_host), fp32
 *           [t][n_out] row-major, 4-byte aligned; it is overwritten (not
 *           accumulated) and must not overlap x or any other job's y. */
typedef struct {
  const il_weight* w;
  int64_t n_out;
  float* y;
} il_job;

/* Cumulative counters (the page's `Backend::stats`, as numbers). */
typedef struct {
  uint64_t uploads;           /* successful il_upload_weight calls        */
  uint64_t upload_bytes;      /* host bytes uploaded (WeightRef::bytes)   */
  uint64_t batches;           /* successful il_matmul_batch* calls        */
  uint64_t jobs;              /* jobs in those batches                    */
  uint64_t launches;          /* kernels launched by those batches        */
  uint64_t weight_bytes;      /* weight bytes those batches streamed      */
  uint64_t flops;             /* 2 * t * n_in * rows summed over jobs     */
  uint64_t errors;            /* calls that returned an error             */
  uint64_t profiled_batches;  /* IL_PROFILE=1: calls whose device time is in device_ns */
  uint64_t device_ns;         /* IL_PROFILE=1: their summed device time (ns)           */
} il_stats;

/*
 * il_upload_weight -- oxinfer src/gpu.rs, `Backend::upload` ("prepares
 * device-side state for a weight matrix").
 *   format   : il_format.
 *   host_ptr : HOST pointer to the weight in the host layout above; only read
 *              during the call (it is copied, then repacked on the device).
 *              Q8/Q4 scales are read with 4-byte loads from the host copy, so
 *              any alignment is accepted.
 *   n_out    : rows, 1 <= n_out <= 2^31 - 1.
 *   n_in     : columns, 1 <= n_in <= 32768; a multiple of 8 for IL_BF16 and of
 *              32 for IL_Q8 / IL_Q4.
 * Returns a new handle, or NULL on error (il_last_error() says why).
 * Synchronous: when it returns the packed weight is resident in HBM.
 */
il_weight* il_upload_weight(int format, const void* host_ptr, int64_t n_out, int64_t n_in);

/*
 * il_matmul_batch -- oxinfer src/gpu.rs, `Backend::matmul` ("runs a batch of
 * matmuls over one shared input in a single submission").
 *   x      : DEVICE pointer, fp32 [t][n_in] row-major, 16-byte aligned.
 *   t      : tokens, 0 <= t <= 2^20.  t == 0 is a successful no-op.
 *   n_in   : must equal every job's handle n_in.
 *   jobs   : HOST array of n_jobs il_job (read during the call only).
 *   n_jobs : 0 <= n_jobs <= 4096; 0 is a successful no-op.
 *   stream : cudaStream_t to enqueue on (NULL = legacy default stream).
 * All arguments are validated, and every launch of the batch is worked out in
 * full (plans, tensor maps, scratch), before anything is launched; on any such
 * error the call returns a negative il_status with no kernel enqueued and no y
 * written.  Only a launch that the CUDA runtime itself rejects (IL_ERR_CUDA,
 * "launch") can leave the earlier launches of the batch enqueued.  On success
 * the work is enqueued asynchronously on `stream`; x, y and the handles must
 * stay valid until it completes.
 * Kernels: small t runs the grouped decode kernels, each weight byte streamed
 * once: t <= 8 for bf16 weights, t <= 16 for Q8/Q4.  Larger t casts x to bf16
 * once and runs the tensor-core kernel (Q8/Q4 weights dequantised to bf16 in
 * shared memory, bf16(fp32(d*q))).  One launch covers every job of one format,
 * up to 32 jobs on a decode kernel and 8 jobs on the tensor-core kernel; a batch
 * beyond those counts, or with several formats, takes one launch per group.
 * Scratch: the tensor-core path keeps a bf16 copy of x and a split-K workspace
 * per (device, stream), owned by the library.  They grow with the stream-ordered
 * allocator (cudaMallocAsync / cudaFreeAsync on `stream`), so growing never
 * waits for the stream; they cannot grow while `stream` is being captured
 * (IL_ERR_UNSUPPORTED): run one call of the largest size on the stream before
 * capturing it.  il_release_scratch frees them.
 * Graphs: a captured call of any entry point uses the scratch of the stream it was captured
 * on, wherever its graph is replayed.  Replays of graphs captured on one stream, and calls
 * on that stream, must therefore not overlap (nothing detects it, and the results would be
 * wrong); capture graphs that are to run side by side on streams of their own.  Scratch that
 * grows after the capture (a larger call on the stream) and il_release_scratch leave the graph
 * without its memory: capture it again before the next replay.
 */
int il_matmul_batch(const float* x, int64_t t, int64_t n_in, const il_job* jobs, int n_jobs,
                    void* stream);

/*
 * il_matmul_batch_host -- il_matmul_batch on HOST buffers, the form in which
 * the pages' `Backend::matmul` takes them (oxinfer src/gpu.rs: `x: &[f32]`,
 * and each `Job` holds `y: &mut [f32]`).
 *   x      : HOST pointer, fp32 [t][n_in] row-major (any alignment).
 *   jobs   : as for il_matmul_batch, but every y is a HOST pointer, fp32
 *            [t][n_out] row-major, 4-byte aligned, overwritten.
 *   t, n_in, n_jobs, stream : as for il_matmul_batch.
 * Host memory may be page-locked (cudaHostAlloc, cudaHostRegister, a pinned
 * torch tensor), pageable or managed; a device pointer for x or a y is
 * rejected with IL_ERR_ARG.  Page-locked buffers are used in place: the kernels
 * read x and write y through their mapped device addresses (over NVLink-C2C on
 * GB300), with no copy operation (a page-locked x that is not 16-byte aligned is
 * copied as below).  Other buffers go through a library-owned device buffer:
 * one copy of x in before the launches, and after them one device->host copy
 * per run of y buffers (y buffers that follow one another in host memory, each
 * starting where the previous one ends, come back in one copy).  Everything is
 * enqueued on `stream` and the call returns once it is; y holds the results
 * after `stream` has completed that work (e.g. cudaStreamSynchronize), and x and
 * y must stay valid, x unchanged, until then.  With page-locked memory nothing
 * blocks the calling thread; with pageable memory the copies behave as
 * cudaMemcpyAsync does for it (the copy of y waits for the kernels).
 * Validation and launch preparation happen before anything is enqueued, with
 * the same rule as il_matmul_batch: an error returns a negative il_status with
 * nothing enqueued, except a copy or launch that the CUDA runtime itself
 * rejects (IL_ERR_CUDA) after earlier work of the call was enqueued.  The
 * device buffer of x and y is scratch per (device, stream), grown and freed
 * like the bf16 copy of x (not during stream capture; il_release_scratch).
 */
int il_matmul_batch_host(const float* x, int64_t t, int64_t n_in, const il_job* jobs, int n_jobs,
                         void* stream);

/*
 * il_matmul_batch_noalloc -- the pages have no counterpart of this entry point.
 * Same arguments and checks as il_matmul_batch, the same split over the decode
 * and tensor-core kernels, results equal to il_matmul_batch's within the
 * per-element tolerance (the tensor-core launches here split K only where the
 * two slices of a tile can run as a CTA pair, which needs no workspace), and
 * the same rule that an error enqueues nothing -- but it never allocates
 * device memory: for callers that cannot let a library call cudaMalloc, such
 * as services that give all device memory to their own pool at start-up, or
 * latency-critical threads for which cudaMalloc / cudaFree may block and
 * synchronise the device.
 *   - The bf16 copy of x used by the tensor-core path (t >= 9 with bf16
 *     weights, t >= 17 with Q8/Q4 weights) goes to a fixed 16 MiB device array
 *     inside the library, held by every GPU that loads the library until the
 *     process exits.  A batch needing more, t * round_up(n_in, 256) * 2 bytes
 *     > 16 MiB, is rejected with IL_ERR_UNSUPPORTED (e.g. t = 2048 fits at
 *     n_in = 4096, not at 12288).
 *   - The Q8/Q4 decode kernel's partial sums of tiles whose K it splits over
 *     CTAs go to a fixed 4 MiB device array (with their arrival counters); a
 *     batch whose plan would need more splits K less.
 *   - The first call on a device looks up the arrays' device addresses and
 *     clears the library's status word and counters there, asynchronously on `stream`; make
 *     that first call before any stream capture.
 *   - Every call shares the same arrays: calls that overlap on the GPU (on
 *     different streams, or from different threads) race and may corrupt each
 *     other's results.  Serialise them, e.g. on one stream.
 *   - A device-side wait that gives up records its code in that status word
 *     and ends the kernel early; il_check_device_status reports it.
 */
int il_matmul_batch_noalloc(const float* x, int64_t t, int64_t n_in, const il_job* jobs, int n_jobs,
                            void* stream);

/*
 * il_upload_gate_up -- a fused gate+up weight.  The pages run the gate and up
 * projections as one shared-input batch and pass the two results straight to
 * gelu_mul (oxinfer 0.0.1, src/drafter.rs, `Drafter::step`: `matmul_multi` over
 * gate and up, then `gelu_mul(&mut g, &u)`).  A handle made here computes that
 * pair and the activation in one job:
 *     h[t][n_out] = gelu(x * Wg^T) * (x * Wu^T)        (elementwise)
 * with gelu the tanh form of the Gemma family the pages serve,
 *     gelu(g) = 0.5 * g * (1 + tanh(sqrt(2/pi) * (g + 0.044715 * g^3))).
 * The pages do not print gelu_mul; this is the reading the library takes.
 *   format            : il_format of BOTH weights.
 *   gate_ptr, up_ptr  : HOST pointers, each one weight in the host layout of
 *                       il_upload_weight with the same n_out and n_in; read
 *                       during the call only.
 *   n_out, n_in       : as for il_upload_weight (n_out = width of h).
 * Returns a handle, or NULL on error.  A job of this handle in il_matmul_batch
 * (or il_matmul_batch_noalloc) takes n_out = the width of h and y = h
 * [t][n_out]; it can share a batch with plain jobs.  Inside, the two weights
 * are stored as one matrix of 2*n_out rows, row 2r = gate row r and row 2r+1 =
 * up row r, so every kernel finds a pair in adjacent rows.  il_weight_bytes
 * gives the sum of both weights' bytes; il_weight_info the format, n_out (the
 * width of h) and n_in; il_dequantize_weight writes the interleaved
 * [2*n_out][n_in] matrix.
 */
il_weight* il_upload_gate_up(int format, const void* gate_ptr, const void* up_ptr, int64_t n_out,
                             int64_t n_in);

/*
 * il_centroid_head -- centroid-masked LM head (oxinfer 0.0.1, src/drafter.rs,
 * end of `Drafter::step`): centroid logits cl = centroids * x, the top_k
 * centroids, the exact logits of the tokens of their clusters, and the token
 * of the first maximum.
 *   x          : DEVICE fp32 [h] (one token), 16-byte aligned.
 *   h          : width; must equal both handles' n_in (<= 32768).
 *   centroids  : bf16 handle [n_cent][h], 1 <= n_cent <= 16384 (a plain weight).
 *   embed      : bf16 handle [vocab][h], vocab a multiple of n_cent; cluster c
 *                owns the tokens ordering[c*per .. (c+1)*per), per = vocab / n_cent.
 *   ordering   : DEVICE u32 [vocab].  An entry >= vocab is skipped (never wins)
 *                and flagged in the device status word (see below).
 *   top_k      : >= 1; k = min(top_k, n_cent) clusters are scored.
 *   token_out  : DEVICE u32 [1]: the winning token id.
 *   score_out  : DEVICE fp32 [1] or NULL: its logit.
 *   selected_out : DEVICE u32 [k] or NULL: the selected centroids in rank order.
 *   scores_out : DEVICE fp32 [k*per] or NULL: every scored logit, index i*per + j
 *                for the j-th token of the i-th selected cluster.
 *   stream     : cudaStream_t (NULL = legacy default stream).
 * Order and ties (the page selects with an unstable partition and scans with a
 * strict '>'; this is the reading taken): centroids rank by larger logit, NaN
 * last, ties to the lower index, and are scanned in that order; among equal
 * logits the first in (rank, position) order wins; NaN and -inf never win, and
 * with no winner the token is 0 and the score -inf.  Logits are fp32 sums of
 * bf16 * fp32 products.  Asynchronous; three kernel launches (the centroid
 * logits run as a one-job il_matmul_batch and are counted as a batch).  Calls
 * on one stream are ordered; the library keeps per-stream scratch for it.
 * An out-of-range ordering entry sets the status word, and il_check_device_status
 * then returns IL_ERR_ARG.
 */
int il_centroid_head(const float* x, int64_t h, const il_weight* centroids, const il_weight* embed,
                     const uint32_t* ordering, int64_t top_k, uint32_t* token_out, float* score_out,
                     uint32_t* selected_out, float* scores_out, void* stream);

/* ---------------------------------------------------------------------------
 * Paged K/V cache: what a decode step does between its q/k/v batch and its
 * output projection.  The pages leave attention outside the matmul backend;
 * these entry points take the batch's fp32 results (q, k, v) and give the fp32
 * x of the next batch, on the same stream, without a copy or a host round trip:
 *     il_kv_extend  block tables and slot maps from the sequences' lengths
 *     il_kv_append  k and v rows into the cache (and il_kv_read back)
 *     il_kv_attend  one new token's attention over each sequence's cache (il_kv_attend_scored:
 *                   with capped or biased logits, or from a later token on)
 *     il_kv_weigh   the attention that each cached token collects
 *     il_kv_evict   sequences cut to the tokens that collected most
 * The cache is the caller's memory, described by value: n_pages pages of
 * page_size tokens.  A token's slot is page * page_size + its index in the page;
 * a sequence's block table lists its pages, so that its position p is in page
 * table[p / page_size].  All pointers are DEVICE pointers; every call is one
 * kernel launch (il_kv_evict one or two; none for an empty call), asynchronous on `stream`,
 * and can be captured in a CUDA graph.  Lengths, tables and slots live on the device and may
 * change between the replays of a graph.  Arguments that only the device can
 * see are checked there: a page or slot outside the cache is never accessed;
 * it is skipped and flagged, and il_check_device_status then returns IL_ERR_ARG.
 * These calls count in il_stats only where they return an error.
 * ------------------------------------------------------------------------- */

/* A paged cache.
 *   format   : IL_BF16, or IL_Q8 as the weights have it: int8 q and one fp32 scale
 *              d per 32 elements of head_dim, value fp32(d*q), or IL_A4: u of 0 .. 15, two per
 *              byte, element 2k in bits 0-3 of byte k, and one pair of bf16 {d, m} per 32 elements,
 *              value fp32(d*u + m).  (The weights' Q4 has no offset; the channels of K seldom lie
 *              about 0.)  Half the bytes of IL_Q8 are not half the time: with up to 4 query heads a K/V
 *              head attention takes 0.73 to 0.77 of it, with 8 or 16 it takes 1.05 to 1.19 times as long.
 *   page_size: tokens per page, 1 .. 2^20.      n_pages: 1 .., n_pages * page_size < 2^31.
 *   n_heads  : K/V heads, 1 .. 1024.
 *   head_dim : 8 .. 256, a multiple of 8 (IL_BF16) or of 32 (IL_Q8, IL_A4).
 *   k, v     : bf16 or int8 elements, or bytes of two; (page, token, head, i) is at
 *              page*page_stride + token*token_stride + head*head_stride + i (IL_A4: strides in
 *              bytes, and i / 2).  Any order of the three strides (64-bit offsets); 16-byte aligned
 *              rows: base address and strides times the element size are multiples of 16.
 *   k_scale, v_scale : IL_Q8: fp32 scales, (page, token, head, i / 32) likewise with
 *              the scale_ strides, in floats (4-byte alignment); IL_A4: the pairs, 4 bytes each
 *              with d in the lower half, in their place; NULL for IL_BF16.
 * Strides of a dimension of extent 1 are not used; the others are at least a
 * row (head_dim, IL_A4 head_dim / 2; scales: head_dim / 32).  Elements must not overlap. */
typedef struct {
  int32_t format;
  int32_t page_size;
  int64_t n_pages;
  int32_t n_heads;
  int32_t head_dim;
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride, token_stride, head_stride;
  int64_t scale_page_stride, scale_token_stride, scale_head_stride;
} il_kv;

/*
 * il_kv_extend -- one scheduler step: sequence r of length lens[r] grows by
 * add[r] tokens, or loses its last -add[r] tokens where add[r] < 0 (rejected draft
 * tokens; add = -lens or less: a finished sequence).  Pages come from and go back to
 * a ring of free pages: cursor = {head, tail} counts the pages ever taken and ever
 * given; entry p is ring[p % ring_size] and the tail - head entries from head are free.
 * Pages are taken in order of sequence, then of position; pages given back follow
 * at the tail in that order, and are free from the next call on.  The table keeps its
 * entries beyond a sequence's pages as they are.
 *   n_seq, page_size : 0 <= n_seq <= 65536; 0 is a successful no-op.
 *   lens, add        : int32 [n_seq] (negative lens count as 0).
 *   table            : int32 [n_seq][table_width], rows table_stride apart; updated.
 *   ring, ring_size  : int32 [ring_size], at least as many as there are pages; updated.
 *   cursor           : int64 [2].
 *   lens_out, cursor_out : the state after the call; may be lens and cursor.
 *   slots            : int32 [max_slots]: slots of the new tokens, sequence by sequence;
 *                      -1 behind the last.      positions: their positions, likewise, or NULL.
 *   first            : int32 [n_seq + 1] or NULL: index in slots of each sequence's first new
 *                      token, and their number.
 *   info             : int64 [4] or NULL: {code, new tokens, pages taken, pages given}.
 * Pages in the ring and the table are not accessed here and move as they are.  A new token in
 * one that no cache has (negative, or with the token's slot at 2^31 - 1 or more) gets the
 * slot 2^31 - 1, which il_kv_append and il_kv_read skip and flag.
 * All or nothing: where there are too few free pages (code bit 0), a sequence
 * would need more pages than table_width (bit 1), the new tokens are more than
 * max_slots (bit 2) or the ring's state is impossible (bit 3), nothing changes: table and ring stay,
 * lens_out = lens, cursor_out = cursor, slots, positions are -1, first is 0, and info
 * has the numbers that were asked for.  The outputs must not overlap each other or
 * an input, except lens_out == lens and cursor_out == cursor.
 */
int il_kv_extend(int64_t n_seq, int64_t page_size, const int32_t* lens, const int32_t* add, int32_t* table,
                 int64_t table_stride, int64_t table_width, int32_t* ring, int64_t ring_size, const int64_t* cursor,
                 int32_t* lens_out, int64_t* cursor_out, int32_t* slots, int64_t max_slots, int32_t* positions,
                 int32_t* first, int64_t* info, void* stream);

/*
 * il_kv_append -- writes n tokens' K and V rows into the cache.
 *   k, v   : fp32, row (token, head) at token*k_stride (v_stride) + head*head_dim; 16-byte
 *            aligned, strides multiples of 4 and at least n_heads*head_dim (e.g. the y
 *            of a k job, or columns of a wider y).
 *   slots  : int32 [n]; a negative slot is skipped.  Slots of one call must differ.
 * bf16 rounds to nearest even.  Q8: d = max|w| / 127 over the 32 elements, q = w / d
 * rounded to nearest even (IEEE divisions, as the weights' test quantiser); a block of
 * zeros has d = 0, q = 0; a block with a NaN or an infinity reads back as NaN.
 * IL_A4: m is the least of the 32 elements rounded down to bf16, d = (max - m) / 15 rounded up
 * to bf16, u = (w - m) / d rounded to nearest even and cut to 0 .. 15 (IEEE single operations
 * each); u = 0 where d = 0, and a block with a NaN, an infinity or a range beyond bf16 reads back
 * as NaN.  A value is off by at most d / 2 and a rounding; d is at most
 * (1 + 2^-7) ((max - min) + 2^-7 |min|) / 15.
 */
int il_kv_append(const il_kv* kv, const float* k, int64_t k_stride, const float* v, int64_t v_stride,
                 const int32_t* slots, int64_t n, void* stream);

/*
 * il_kv_read -- the inverse of il_kv_append: the cached values of n slots as fp32 (exact
 * for bf16, fp32(d*q) for Q8, fp32(d*u + m) for A4), rows of a negative slot as zeros.  k, v as above, written.
 */
int il_kv_read(const il_kv* kv, const int32_t* slots, int64_t n, float* k, int64_t k_stride, float* v,
               int64_t v_stride, void* stream);

/*
 * il_kv_attend -- attention of one token per sequence over its cached tokens:
 *     s_t = scale * q_h . k_t,   out_h = sum_t softmax(s)_t v_t,   lse_h = ln sum_t exp(s_t)
 * over t in [max(0, len - window), len), query head h reading K/V head
 * h / (n_q_heads / n_heads).  The new token itself is one of the len (append it first).
 *   q      : fp32 [n_seq][n_q_heads][head_dim], sequences q_stride apart; 16-byte aligned,
 *            q_stride a multiple of 4.         out: likewise with out_stride, overwritten; apart
 *            from q, or columns of the same buffer beside it.
 *   lse    : fp32 [n_seq][n_q_heads] or NULL.
 *   table, table_stride, table_width, lens : as il_kv_extend leaves them.  A length is cut to
 *            0 .. table_width * page_size.
 *   n_q_heads : a multiple of the cache's n_heads, at most 32768.    n_seq: 0 .. 65536.
 *   window : tokens seen, counted from the end; 0: all.
 * A sequence of length 0 gives out = 0 and lse = -inf.  Cached values outside the
 * attended range are never used, NaN or not.  q, K and V that are attended must be finite:
 * where one is not, that sequence's heads that read it give NaN or infinity, of V in its column
 * (Q8, A4: in its block's 32) alone.  Nor may len times the largest |V| reach 2^127 (A4: 2^103, since
 * its sums may be kept 2^24 times as large): the sums of p V are divided at the end.  Work is split
 * over the length and joined in an order that depends on the lengths only, so that equal
 * calls give equal bits.
 * Rounding: sums and softmax statistics are fp32.  Over a bf16 cache q and the weights p keep
 * 21 or more of their 24 bits.  Over a Q8 cache an element of q keeps 22 bits, or 2^-38 of its
 * head's largest where that is coarser.  A weight p there multiplies V's scale d, in tiles of 16
 * or 32 tokens; p below is relative to the tile's largest, or to 2^-24 of the sequence's largest so
 * far where that is more.  p d keeps 22 bits, or 2^-26 d where that is coarser.  In a tile with p below
 * 2^-26 or d below 2^-12 of the sequence's largest so far, the second bound is 2^-12 of p times the
 * tile's largest d of the same 32 columns instead, and p below 2^-104 counts as 0.  Over an A4 cache,
 * and with il_kv_attend_scored over a Q8 one, an element of q keeps 22 bits, or 2^-49 of its head's
 * largest where that is coarser, and p d keeps 22 bits, or 2^-49 of the sequence's largest so far; in
 * a tile with p below 2^-26 or d below 2^-12 of those, 22 bits down to 2^-104 of it, where it counts
 * as 0.
 * Workspace: il_kv_extend and il_kv_attend share one of about 5 MB per (device, stream), owned by the library,
 * allocated (stream-ordered) by the first of these calls on the stream and never moved: run one before
 * capturing the stream (IL_ERR_UNSUPPORTED otherwise).  il_release_scratch frees it.  A graph keeps using
 * the workspace of the stream it was captured on: see "Graphs" at il_matmul_batch.
 */
int il_kv_attend(const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                 int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale,
                 int64_t window, float* out, int64_t out_stride, float* lse, void* stream);

/* What il_kv_attend_scored does to a logit, scale q_h . k_t at first; all of it zero or NULL: nothing.
 *   cap       : > 0: s = cap tanh(s / cap).
 *   slopes    : fp32 [n_q_heads] or NULL: then s += slopes[h] (pos_t - pos_last), a bias that grows
 *               with the distance from the sequence's last token.
 *   starts    : int32 [n_seq] or NULL: tokens of index below starts[r] are not seen (the first token
 *               of the document that the new token belongs to); negative: all are, len or more: none is.
 *   positions : int32 [n_seq][positions_width], rows positions_stride apart, or NULL (a token's
 *               position is its index): positions of the tokens where il_kv_evict has moved them.
 *               A length is cut to positions_width.  Only the bias goes by them: window and starts count
 *               indices, which say nothing about a token's place once something was evicted.  Do not
 *               combine those with an eviction; its `recent` stands in for a window.
 * cap is 0 or 2^-100 to 2^100; scale / cap, an element of q times that, and slopes must be finite. */
typedef struct {
  float cap;
  const float* slopes;
  const int32_t* starts;
  const int32_t* positions;
  int64_t positions_stride, positions_width;
} il_kv_score;

/*
 * il_kv_attend_scored -- il_kv_attend with capped and biased logits and sequences that begin later.
 * The window counts by index; with starts, a token is seen that both allow.  A sequence of which no
 * token is seen gives out = 0 and lse = -inf.  The cap and the bias are fp32: a logit's error is that
 * of tanhf and three roundings times cap, and three of the bias (log2(e), the slope times it, the sum).
 */
int il_kv_attend_scored(const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                        int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale,
                        int64_t window, const il_kv_score* score, float* out, int64_t out_stride, float* lse,
                        void* stream);

/*
 * il_kv_weigh -- what each cached token collects of one new token's attention, over all query heads:
 *     weights_out[r][t] = (t is new ? 0 : weights[r][t]) + sum_h exp(s_t - lse_h)
 * for t < lens[r], with s as il_kv_attend (or, with score, il_kv_attend_scored) has it; tokens that
 * are not seen add nothing.  Call it with the same arguments, and that call's lse.  K is read, V is not.
 *   q .. score : as for il_kv_attend_scored; score may be NULL.
 *   lse       : fp32 [n_seq][n_q_heads].
 *   add       : int32 [n_seq] or NULL: the last add[r] tokens are new, whatever weights holds there
 *               (il_kv_extend's add; all of them for a new sequence; negative: none).
 *   weights, weights_out : fp32 [n_seq][weights_width], rows weights_stride apart; may be the same.
 *               A length is cut to weights_width (at most 2^30).  Entries from the length on are left
 *               as they are.
 * Sums are fp32, in an order that depends on the lengths only: equal calls give equal bits.  K, q and
 * lse that are read must be finite.  Needs no workspace.
 */
int il_kv_weigh(const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale,
                int64_t window, const il_kv_score* score, const float* lse, const int32_t* add, const float* weights,
                float* weights_out, int64_t weights_stride, int64_t weights_width, void* stream);

/*
 * il_kv_evict -- cuts sequences longer than `keep` to that many tokens: those at the first positions,
 * the most recent ones and, of the others, those of the largest weight (of equal ones those of the
 * lower index; NaN counts as the least).  Kept tokens of index keep and more move to the places of
 * tokens before it that go, the i-th to the i-th; the others stay where they are, so that a token's
 * index no longer tells its position (hence `positions`).  Sequences of up to `keep` tokens stay as
 * they are.  lens, table and the free pages stay too: drop holds the changes of length for
 * il_kv_extend's add, which gives the pages back -- once, where the caches of several layers share a
 * table and each has been cut by a call of its own.
 * What goes by index goes wrong once tokens were moved: a window and starts (il_kv_score), and an add below 0
 * for a rejected draft, which drops the last indices -- take drafts back before the eviction.
 *   keep      : 1 to 2^30.     first, recent : tokens of position below first, or above that of the
 *               last token less recent, stay whatever their weight; first + recent <= keep.
 *   weights, weights_out : as for il_kv_weigh; the weights move with their tokens.
 *   positions, positions_out : int32 likewise [n_seq][positions_width], not negative, distinct in a
 *               sequence and the last token's the newest; both NULL: a token's position is its index
 *               (right until something was evicted).  A length is cut to their width.  The caller writes those of new tokens (il_kv_extend's
 *               positions are indices).  After an eviction the last token is seldom the newest: cut a sequence
 *               again only when a new token has come.
 *   kept      : int32 [n_seq][keep], rows kept_stride apart: the index that a token now at i had, -1
 *               from the new length on.
 *   drop      : int32 [n_seq]: the new length less lens[r] (of a length that was cut, all that is
 *               beyond goes too).
 * The pages of a sequence that is cut must be its own.  Outputs must not overlap each other or an
 * input, except weights_out == weights and positions_out == positions.  One launch where rows are at
 * most keep + 64 wide, else two; needs no workspace.
 */
int il_kv_evict(const il_kv* kv, const int32_t* table, int64_t table_stride, int64_t table_width, const int32_t* lens,
                int64_t n_seq, int64_t keep, int64_t first, int64_t recent, const float* weights, float* weights_out,
                int64_t weights_stride, int64_t weights_width, const int32_t* positions, int32_t* positions_out,
                int64_t positions_stride, int64_t positions_width, int32_t* kept, int64_t kept_stride, int32_t* drop,
                void* stream);

/* 1 if the handle came from il_upload_gate_up, 0 if from il_upload_weight,
 * -1 for an invalid handle. */
int il_weight_is_gate_up(const il_weight* w);

/* Releases a handle and its device memory (synchronises the device).
 * NULL is ignored; an unknown pointer is ignored and counted as an error. */
void il_free_weight(il_weight* w);

/* Host-layout byte size of the weight, oxinfer src/gpu.rs `WeightRef::bytes`:
 * 2*n_out*n_in (bf16), n_out*n_in*9/8 (Q8), n_out*n_in*5/8 (Q4).  -1 for an
 * invalid handle. */
int64_t il_weight_bytes(const il_weight* w);

/* Format and shape of a handle (for a gate+up handle, n_out is the width of
 * h).  Any out pointer may be NULL. */
int il_weight_info(const il_weight* w, int* format, int64_t* n_out, int64_t* n_in);

/*
 * il_dequantize_weight -- test hook: writes every element of the uploaded
 * weight as fp32 to dev_out [n_out][n_in] (DEVICE pointer, 4-byte aligned),
 * reading the packed device layout with the same element decoders the matmul
 * kernels use.  bf16 widens exactly; Q8/Q4 give fp32(d*q).  Asynchronous on
 * `stream`.  For a gate+up handle dev_out is [2*n_out][n_in], rows interleaved
 * as described at il_upload_gate_up.
 */
int il_dequantize_weight(const il_weight* w, float* dev_out, void* stream);

/* Reads (and clears) the device-side status words that bounded waits in the
 * kernels set when they give up -- the one of il_matmul_batch and
 * il_centroid_head, and the one of il_matmul_batch_noalloc -- on the current
 * device.  Synchronises `stream`.  Returns IL_OK, or IL_ERR_DEVICE_TIMEOUT if a
 * wait timed out since the last call; in that case it also waits for the
 * device and clears the library's split-K workspaces on it, so that later
 * batches start from a clean state.  Returns IL_ERR_ARG if no wait timed out
 * but il_centroid_head met an ordering entry >= vocab, or an il_kv_* call a page
 * or slot outside its cache. */
int il_check_device_status(void* stream);

/* Frees the scratch the library keeps for `stream` on the current device (the
 * bf16 copy of x, the split-K workspace, the LM-head scratch, the device copies
 * of x and y of il_matmul_batch_host, the K/V workspace), in stream order:
 * call it before destroying a stream the library has run on (for
 * cudaStreamPerThread on the thread itself, before it ends).  Graphs captured on the
 * stream must not be replayed any more.  A later call on
 * the stream allocates afresh.  Returns IL_OK or IL_ERR_CUDA. */
int il_release_scratch(void* stream);

/* Message of the last error on this thread ("" if none). */
const char* il_last_error(void);

/* il_status of the last error on this thread (IL_OK if none); useful after
 * il_upload_weight returned NULL.  Each entry point clears it on entry. */
int il_last_status(void);

/* Copies the cumulative counters into *out (the page's `Backend::stats`, a
 * cumulative timing summary when profiling).  With IL_PROFILE=1 in the
 * environment, il_matmul_batch, il_matmul_batch_host (its launches, not its
 * copies) and il_centroid_head record a CUDA event before and after their
 * launches on their stream (not while the stream is being
 * captured, and not il_matmul_batch_noalloc); il_get_stats then waits for every
 * recorded call to finish and adds its device time to device_ns.  Without
 * IL_PROFILE nothing is recorded and nothing waits.  The entry points also mark
 * their host work with NVTX ranges, which cost nothing unless a tool listens. */
int il_get_stats(il_stats* out);
/* Zeroes the counters (with IL_PROFILE=1, after waiting for the recorded calls). */
void il_reset_stats(void);

/* IL_VERSION of the loaded library. */
int il_version(void);

#ifdef __cplusplus
}
#endif

#endif /* IL_H_ */
