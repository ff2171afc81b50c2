/*
 * qar.h -- C ABI of libqar: dynamic block-wise int8 quantization and
 * quantized reduction, one GPU's share of a quantized AllReduce, for AMD
 * Instinct MI355X (gfx950).
 *
 * The method is EQuARX ("EQuARX: Efficient Quantized AllReduce in XLA for
 * Distributed Machine Learning Acceleration"; page summary, section
 * "technical framework", steps 1-4; section "key design", item 1): the
 * tensor is cut into blocks, each block is quantized from BF16/FP32 to INT8
 * with a range found at run time, the AllReduce sums the quantized
 * contributions, and the result is dequantized back to the original type.
 * The pages leave the arithmetic open; libqar fixes it as follows, for every
 * call, bit for bit:
 *
 *   scale  s   = absmax / 127            one IEEE binary32 division
 *   code   q_i = 0 if s == 0, else clamp(rne(x_i / s), -127, 127)
 *                (x_i / s is the correctly rounded binary32 quotient; rne
 *                rounds to the nearest integer, ties to even; -128 is
 *                never produced)
 *   value  y_i = (float)q_i * s           one binary32 multiply
 *   bf16   round-to-nearest-even of the binary32 value
 *
 * All binary32 arithmetic rounds to nearest even with gradual underflow (no
 * flush to zero); multiplies and adds are never fused.
 *
 * Layout.  A buffer of n elements is nb = n / block consecutive blocks of
 * `block` elements (row-major flattening; for a [rows, hidden] tensor with
 * hidden % block == 0 the blocks run along the hidden dimension).  Codes are
 * int8[n] in element order; scales are a separate float[nb], one per block,
 * in block order.
 *
 * Conventions shared by every call:
 *   - Pointers are device pointers owned by the caller.  libqar never
 *     allocates, frees or synchronizes device memory at run time (its one
 *     static device array, the workspace of qar_allreduce_simulated_static,
 *     is part of the loaded code object).
 *   - Calls are asynchronous: work is enqueued on `stream` (a hipStream_t
 *     passed as void*; NULL is the default stream) and the call returns.
 *   - Arguments are checked before anything is enqueued.  A failed check
 *     returns a QAR_ERR_* status and enqueues nothing.  A failed launch
 *     returns QAR_ERR_HIP; qar_last_error() then names the HIP error.
 *   - n == 0 is a valid empty call: QAR_OK, nothing enqueued, no pointer is
 *     read.
 *   - Requirements (calls with a block argument): block is 64, 128 or 256;
 *     n % block == 0;
 *     n <= QAR_MAX_ELEMENTS; element and code pointers 16-byte aligned;
 *     scale pointers 4-byte aligned.
 *   - Inputs must be finite, and so must every binary32 sum a reduce or
 *     ring step forms (the sum of finite values can overflow).  Output for
 *     NaN or infinite input, or for an overflowed sum, is unspecified (it is
 *     not checked, for speed).
 *   - Output buffers must not overlap input buffers, except where a call
 *     says otherwise.  Partial overlap is rejected with QAR_ERR_INVALID_ARG.
 *   - Any block-aligned sub-range of a valid call (pointers advanced by
 *     k*block elements and k scales) is itself a valid call with the same
 *     results in that range.
 *   - Thread-safe.  Global state: the per-thread text behind
 *     qar_last_error(); a per-device pool of HIP events that the calls
 *     forking work onto side streams borrow while they enqueue (created on
 *     demand, one set per call in flight at once, never device memory); and
 *     the static workspace of qar_allreduce_simulated_static.
 */
#ifndef QAR_H
#define QAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The enums below are passed by value across the ABI.  A C caller may pass
 * any int in their place; compiled as C++ (the library itself) they take int
 * as their fixed underlying type, so every such value is a value of the type
 * and an unknown one reaches the argument checks (QAR_ERR_UNSUPPORTED or
 * QAR_ERR_INVALID_ARG) instead of being undefined before them.  In C an
 * enum is an int-sized integer type either way. */
#ifdef __cplusplus
#define QAR_ENUM_BASE : int
#else
#define QAR_ENUM_BASE
#endif

typedef enum qar_status QAR_ENUM_BASE {
    QAR_OK = 0,
    QAR_ERR_INVALID_ARG = 1, /* null pointer, n % block != 0, bad rank count, overlap */
    QAR_ERR_MISALIGNED = 2,  /* a pointer breaks the alignment rule above */
    QAR_ERR_UNSUPPORTED = 3, /* block size or dtype outside what is built */
    QAR_ERR_HIP = 4,         /* the HIP runtime refused a launch or call */
    QAR_ERR_CAPACITY = 5     /* the call needs more static workspace than QAR_STATIC_WORKSPACE_BYTES */
} qar_status;

typedef enum qar_dtype QAR_ENUM_BASE {
    QAR_BF16 = 0, /* bfloat16, stored as 16-bit patterns */
    QAR_F32 = 1   /* IEEE binary32 */
} qar_dtype;

#define QAR_MAX_RANKS 32
#define QAR_MAX_ELEMENTS ((size_t)1 << 40)
#define QAR_MAX_STREAMS 16

/*
 * Per-block dynamic quantization ("technical framework" steps 1-2; "key
 * design" item 1).
 *   x       [in]  n elements of `dtype`.
 *   codes   [out] int8[n].
 *   scales  [out] float[n / block].
 */
qar_status qar_quantize_blocks(const void* x, qar_dtype dtype, size_t n, uint32_t block,
                               int8_t* codes, float* scales, void* stream);

/*
 * One-shot N-way reduce of quantized contributions, then requantization of
 * the sum ("technical framework" step 3: the AllReduce works on the
 * quantized data; the error that summation builds up is the problem the
 * abstract and the "problem definition" section name).  For each element:
 *   acc = y_0;  acc = acc + y_r for r = 1 .. nranks-1  (binary32, rank order)
 * and the result is quantize(acc) per block.
 *   codes, scales  [in]  HOST arrays of nranks DEVICE pointers, rank order;
 *                        codes[r] is int8[n], scales[r] is float[n/block].
 *   nranks         1 .. QAR_MAX_RANKS.
 *   codes_out      [out] int8[n];  scales_out [out] float[n/block].  These
 *                  may be exactly the buffers of one input rank (in place).
 *   out            [out, optional] NULL, or n elements of out_dtype that
 *                  receive dequantize(codes_out, scales_out) -- step 4,
 *                  fused.  It is the requantized result, not the raw sum, so
 *                  that every rank of a real AllReduce dequantizes identical
 *                  bits.
 */
qar_status qar_reduce_quantized(const int8_t* const* codes, const float* const* scales,
                                uint32_t nranks, size_t n, uint32_t block,
                                int8_t* codes_out, float* scales_out,
                                void* out, qar_dtype out_dtype, void* stream);

/*
 * This rank's quantize fused into the reduce: the one-shot reduce in which
 * rank `own` contributes its unquantized buffer x_own.  x_own is quantized in
 * the same pass ("technical framework" step 2), its codes and scales are
 * written to codes[own] / scales[own] (what the peers receive), and those
 * same values enter the rank-order sum ("technical framework" step 3).
 * Results (codes[own], scales[own], codes_out, scales_out, out) are
 * bit-identical to qar_quantize_blocks(x_own -> codes[own], scales[own])
 * followed by qar_reduce_quantized; x_own is read once and codes[own] is
 * never read back.
 *   x_own        [in]  n elements of dtype (bf16 or fp32).
 *   own          0 .. nranks-1.
 *   codes, scales HOST arrays of nranks DEVICE pointers; entry own is an
 *                output, the others are inputs (as in qar_reduce_quantized).
 *   codes_out, scales_out, out, out_dtype  as in qar_reduce_quantized, but
 *                they may not be rank own's buffers.
 */
qar_status qar_quantize_reduce(const void* x_own, qar_dtype dtype, uint32_t own, int8_t* const* codes,
                               float* const* scales, uint32_t nranks, size_t n, uint32_t block,
                               int8_t* codes_out, float* scales_out, void* out, qar_dtype out_dtype,
                               void* stream);

/* Elements per run of the chunked calls' interleaved chunks. */
#define QAR_CHUNK_RUN_ELEMS (1u << 18)

/*
 * The same reduce as a pipeline of chunks over streams (the pages' deep
 * pipelining of communication and compute, "key innovations" item 2 and
 * "key design" item 3, taken on one GPU).  The elements are taken in runs
 * of QAR_CHUNK_RUN_ELEMS (the last run shorter; a run holds whole blocks)
 * and cut into `nchunks` interleaved chunks: chunk c computes runs c,
 * c + nchunks, c + 2 nchunks, ..., so the chunks that run at once read
 * neighbouring addresses.  Chunk c is enqueued on streams[c % nstreams]
 * behind whatever that stream already holds.  Nothing else is enqueued: no event, no wait.  The caller
 * orders the chunks after the producers of the inputs and before the
 * consumers of the outputs on every stream used (events, or by producing
 * and consuming on those streams).  Consecutive calls on the same streams
 * therefore overlap: a stream holds its chunk in flight and the next
 * call's behind it (double buffering), so one stream's kernel ramps up
 * while another's drains; two calls with the same n, nchunks and streams
 * give chunk c the same runs on the same stream.  Results are
 * bit-identical to qar_reduce_quantized for every nchunks and nstreams.
 *   nchunks   >= 1 (clipped to the number of runs).
 *   streams   HOST array of nstreams hipStream_t (as void*), 1 .. QAR_MAX_STREAMS;
 *             NULL (the default stream) is allowed; the first
 *             min(nchunks, nstreams) are used.
 */
qar_status qar_reduce_quantized_chunked(const int8_t* const* codes, const float* const* scales,
                                        uint32_t nranks, size_t n, uint32_t block,
                                        int8_t* codes_out, float* scales_out,
                                        void* out, qar_dtype out_dtype,
                                        uint32_t nchunks, void* const* streams, uint32_t nstreams);

/*
 * qar_reduce_quantized_chunked ordered as one operation on `stream`: the
 * chunks start after everything already enqueued on `stream`, and `stream`
 * waits for all of them.  A stream of `streams` that is `stream` itself
 * needs no event; every other one costs an event record and a wait at each
 * end of the call (on MI355X with ROCm 7 this fork and join cost tens of
 * microseconds per call, so a sequence of independent reduces is better
 * enqueued with qar_reduce_quantized_chunked between one fork and one
 * join).  The events come from a per-device pool (created on first use,
 * never device memory).  Results are bit-identical to qar_reduce_quantized.
 *   nchunks   >= 1 (clipped to the number of runs of QAR_CHUNK_RUN_ELEMS).
 *   streams   HOST array of nstreams hipStream_t (as void*),
 *             1 .. QAR_MAX_STREAMS; an entry may be NULL (the default
 *             stream) only when `stream` is NULL too, i.e. when it is the
 *             calling stream.
 */
qar_status qar_reduce_quantized_pipelined(const int8_t* const* codes, const float* const* scales,
                                          uint32_t nranks, size_t n, uint32_t block,
                                          int8_t* codes_out, float* scales_out,
                                          void* out, qar_dtype out_dtype,
                                          uint32_t nchunks, void* const* streams,
                                          uint32_t nstreams, void* stream);

/*
 * One ring step: dequantize the incoming quantized buffer, add this rank's
 * own unquantized values, requantize ("technical framework" step 3 taken as
 * a ring; the error accumulates over the N-1 steps):
 *   acc_i = y_in,i + x_local,i   (binary32), then quantize(acc) per block.
 *   codes_in, scales_in  [in]  int8[n], float[n/block].
 *   local                [in]  n elements of `dtype` (bf16 or fp32).
 *   codes_out, scales_out [out] int8[n], float[n/block]; may be exactly
 *                        codes_in / scales_in (in place).
 */
qar_status qar_ring_step(const int8_t* codes_in, const float* scales_in,
                         const void* local, qar_dtype dtype, size_t n, uint32_t block,
                         int8_t* codes_out, float* scales_out, void* stream);

/*
 * Dequantize back to the original type ("technical framework" step 4):
 *   out_i = (float)q_i * s_b, stored as binary32 or rounded to bf16.
 *   codes, scales  [in]  int8[n], float[n/block].
 *   out            [out] n elements of out_dtype.
 */
qar_status qar_dequantize(const int8_t* codes, const float* scales, size_t n, uint32_t block,
                          void* out, qar_dtype out_dtype, void* stream);

/*
 * The comparator the pages measure against: the same N-way reduction on the
 * unquantized data (EQuARX abstract: the 1.8x is over a BF16 AllReduce).
 * For each element the binary32 sum of the ranks' values in rank order,
 * stored in the input type (bf16: rounded to nearest even).
 *   x       [in]  HOST array of nranks DEVICE pointers, each n elements of
 *                 dtype, rank order.
 *   nranks  1 .. QAR_MAX_RANKS.
 *   n       any multiple of 16 (no block structure).
 *   out     [out] n elements of dtype; may be exactly one input buffer.
 */
qar_status qar_reduce_unquantized(const void* const* x, uint32_t nranks, size_t n, qar_dtype dtype,
                                  void* out, void* stream);

/*
 * The whole quantized AllReduce of N rank buffers, simulated on one GPU:
 * the result every rank of a real AllReduce would hold, computed with the
 * calls above ("technical framework" steps 1-4, pipelined over chunks as in
 * "key innovations" item 2).  The buffer is cut into `nchunks` block-aligned
 * chunks; chunk c runs on streams[c % nstreams]:
 *   QAR_SCHEDULE_ONE_SHOT: every rank's chunk is quantized
 *     (codes_work[r], scales_work[r]), then one fused reduce in rank order
 *     0..N-1 requantizes the sum in place into codes_work[0]/scales_work[0]
 *     and writes its dequantized value to out.  The last rank's quantize
 *     runs inside that reduce (qar_quantize_reduce) when N > 1; the results
 *     are the same bits.  With nchunks = N the chunks are the N slices of a
 *     two-shot AllReduce's reduce-scatter (the TACO page, section 2.B
 *     item 3, kernel fusion and overlap: reduce-scatter, then all-gather); its
 *     all-gather forwards the requantized codes unchanged.
 *   QAR_SCHEDULE_RING: chunk c starts at rank s = c mod N, as the chunk
 *     rank s injects first in a ring: quantize(x_s), then ring steps adding
 *     x_{s+1}, ..., x_{s+N-1} (ranks mod N) in place in codes_work[0] /
 *     scales_work[0], then dequantize to out.  With nchunks = N this is the
 *     classic ring's reduce-scatter order; the all-gather forwards codes
 *     unchanged, so it adds no error and is not simulated.
 *   x            [in]  HOST array of nranks DEVICE pointers, n elements of dtype.
 *   codes_work, scales_work  HOST arrays of DEVICE pointers: int8[n] and
 *                float[n/block] workspaces; nranks of each for ONE_SHOT, only
 *                [0] is used for RING (the rest may be NULL).
 *   out          [out] n elements of dtype.
 *   nchunks      >= 1 (clipped to the number of blocks); streams: HOST array
 *                of 1..QAR_MAX_STREAMS handles (NULL only when `stream` is
 *                NULL); `stream` orders the whole call as in
 *                qar_reduce_quantized_pipelined.
 * Results are bit-identical for every nchunks and nstreams under ONE_SHOT;
 * under RING they depend on nchunks through each chunk's starting rank.
 */
typedef enum qar_schedule QAR_ENUM_BASE { QAR_SCHEDULE_ONE_SHOT = 0, QAR_SCHEDULE_RING = 1 } qar_schedule;

qar_status qar_allreduce_simulated(const void* const* x, qar_dtype dtype, uint32_t nranks, size_t n,
                                   uint32_t block, qar_schedule schedule, int8_t* const* codes_work,
                                   float* const* scales_work, void* out, uint32_t nchunks,
                                   void* const* streams, uint32_t nstreams, void* stream);

/*
 * For callers that cannot allocate: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc.  qar_allreduce_simulated
 * with the same arguments minus the workspaces and the side streams: every
 * chunk runs on `stream` in chunk order, and the per-rank code and scale
 * staging lives in a static device array inside libqar,
 * QAR_STATIC_WORKSPACE_BYTES per device, held by every device the library
 * runs on until the process ends.  The call allocates nothing, records no
 * event and synchronizes nothing; results are bit-identical to
 * qar_allreduce_simulated with the same schedule and nchunks.
 *   Capacity: one-shot stages nranks * (n + 4 n/block) bytes, the ring
 *   n + 4 n/block (each rounded up to 256 bytes per rank and array); a
 *   call that needs more returns QAR_ERR_CAPACITY and enqueues nothing
 *   (qar_last_error() gives the sizes).
 *   Sharing: all calls on one device use the same array.  Calls whose work
 *   overlaps in time on one device (on different streams, or from several
 *   threads without ordering between their streams) race on it; order them
 *   on one stream or with events.  Nothing in the array needs to start at
 *   zero: every byte a call reads there was written earlier by that call.
 *   The device address of the array is looked up on the first call per
 *   device (hipGetSymbolAddress) and cached.
 */
#define QAR_STATIC_WORKSPACE_BYTES ((size_t)64 << 20)

qar_status qar_allreduce_simulated_static(const void* const* x, qar_dtype dtype, uint32_t nranks, size_t n,
                                          uint32_t block, qar_schedule schedule, void* out, uint32_t nchunks,
                                          void* stream);

/*
 * Row-bounded blocks: the same four operations on a [rows, row_len] tensor
 * whose block grid restarts at every row, so the last block of a row holds
 * row_len % block elements when row_len is not a multiple of block (a block
 * never spans two rows).  Each row has per_row = ceil(row_len / block)
 * blocks; scales hold rows * per_row values, row-major; codes and data hold
 * rows * row_len elements, row-major.  The arithmetic of every block is that
 * of the calls above, a partial block taking its absmax over its own
 * elements.  When row_len % block == 0 the block grids coincide and the call
 * is exactly the flat call with n = rows * row_len.
 * Requirements: block 64, 128 or 256; rows * row_len <= QAR_MAX_ELEMENTS;
 * rows * per_row <= QAR_MAX_ROW_BLOCKS; data pointers aligned to their
 * element size, scales to 4 bytes, codes unconstrained (the flat fast path
 * is taken when the flat call's 16-byte alignment also holds).
 */
#define QAR_MAX_ROW_BLOCKS ((size_t)1 << 26)

qar_status qar_quantize_rows(const void* x, qar_dtype dtype, size_t rows, size_t row_len, uint32_t block,
                             int8_t* codes, float* scales, void* stream);
qar_status qar_reduce_quantized_rows(const int8_t* const* codes, const float* const* scales, uint32_t nranks,
                                     size_t rows, size_t row_len, uint32_t block, int8_t* codes_out,
                                     float* scales_out, void* out, qar_dtype out_dtype, void* stream);
qar_status qar_ring_step_rows(const int8_t* codes_in, const float* scales_in, const void* local, qar_dtype dtype,
                              size_t rows, size_t row_len, uint32_t block, int8_t* codes_out, float* scales_out,
                              void* stream);
qar_status qar_dequantize_rows(const int8_t* codes, const float* scales, size_t rows, size_t row_len,
                               uint32_t block, void* out, qar_dtype out_dtype, void* stream);

/*
 * FP8 E4M3 codes.  The same calls with 8-bit floating-point codes in place
 * of int8 integers: the format the TACO page argues for ("TACO: Efficient
 * Communication Compression of Intermediate Tensors for Scalable
 * Tensor-Parallel LLM Training", page summary in Dutch, section 2.A "Waarom
 * FP8?", why FP8), with the per-block scale of its section 2.B item 2
 * "Dual-Scale (DS) Quantization" that brings the block into FP8's range Q_max (only
 * that scale; no rotation).  E4M3 is the OCP format: sign, 4 exponent bits
 * with bias 7, 3 mantissa bits, subnormals (m/8) * 2^-6, no infinity, codes
 * 0x7F and 0xFF NaN (never produced), largest finite value 448.
 *
 *   scale  s   = absmax / 448            one IEEE binary32 division
 *   code   c_i = 0x00 if s == 0; else the E4M3 value nearest to
 *                clamp(x_i / s, -448, 448) (the correctly rounded binary32
 *                quotient), ties to the even mantissa; the sign is kept, so
 *                a negative quotient that rounds to zero gives 0x80 (-0)
 *   value  y_i = e4m3(c_i) * s           one binary32 multiply
 *
 * Codes are uint8_t[n], one byte per element, in the same layout as the int8
 * codes; scales, alignment, aliasing, streams and errors are exactly those of
 * the int8 call of the same name.  The reduce, the one-kernel step and the
 * ring step sum in binary32 in rank order and requantize with this
 * quantizer; a sum is -0 only when every term is.
 */
qar_status qar_quantize_blocks_e4m3(const void* x, qar_dtype dtype, size_t n, uint32_t block, uint8_t* codes,
                                    float* scales, void* stream);
qar_status qar_reduce_quantized_e4m3(const uint8_t* const* codes, const float* const* scales, uint32_t nranks,
                                     size_t n, uint32_t block, uint8_t* codes_out, float* scales_out, void* out,
                                     qar_dtype out_dtype, void* stream);
qar_status qar_quantize_reduce_e4m3(const void* x_own, qar_dtype dtype, uint32_t own, uint8_t* const* codes,
                                    float* const* scales, uint32_t nranks, size_t n, uint32_t block,
                                    uint8_t* codes_out, float* scales_out, void* out, qar_dtype out_dtype,
                                    void* stream);
qar_status qar_ring_step_e4m3(const uint8_t* codes_in, const float* scales_in, const void* local,
                              qar_dtype dtype, size_t n, uint32_t block, uint8_t* codes_out, float* scales_out,
                              void* stream);
qar_status qar_dequantize_e4m3(const uint8_t* codes, const float* scales, size_t n, uint32_t block, void* out,
                               qar_dtype out_dtype, void* stream);

/*
 * 4-bit integer codes.  The same calls with 4-bit codes, two per byte.  The
 * pages name 4-bit communication quantization only through titles in their
 * reference lists (SDP4Bit; Echo, error-compensated 4-bit tensor-parallel
 * communication); libqar takes the int8 method at 4 bits:
 *
 *   scale  s   = absmax / 7              one IEEE binary32 division
 *   code   q_i = 0 if s == 0, else clamp(rne(x_i / s), -7, 7)
 *   value  y_i = (float)q_i * s
 *
 * Codes are packed: element 2k in the low nibble of byte k, element 2k+1 in
 * the high nibble, two's complement (-8 is never produced); a buffer of n
 * elements takes n/2 bytes.  A block-aligned sub-range starts block/2 bytes
 * per block into the codes.  Alignment, aliasing (in place: the whole packed
 * buffer and the scales), streams and errors are those of the int8 call of
 * the same name; sizes of code buffers are n/2 bytes instead of n.
 */
qar_status qar_quantize_blocks_int4(const void* x, qar_dtype dtype, size_t n, uint32_t block, uint8_t* codes,
                                    float* scales, void* stream);
qar_status qar_reduce_quantized_int4(const uint8_t* const* codes, const float* const* scales, uint32_t nranks,
                                     size_t n, uint32_t block, uint8_t* codes_out, float* scales_out, void* out,
                                     qar_dtype out_dtype, void* stream);
qar_status qar_quantize_reduce_int4(const void* x_own, qar_dtype dtype, uint32_t own, uint8_t* const* codes,
                                    float* const* scales, uint32_t nranks, size_t n, uint32_t block,
                                    uint8_t* codes_out, float* scales_out, void* out, qar_dtype out_dtype,
                                    void* stream);
qar_status qar_ring_step_int4(const uint8_t* codes_in, const float* scales_in, const void* local,
                              qar_dtype dtype, size_t n, uint32_t block, uint8_t* codes_out, float* scales_out,
                              void* stream);
qar_status qar_dequantize_int4(const uint8_t* codes, const float* scales, size_t n, uint32_t block, void* out,
                               qar_dtype out_dtype, void* stream);

/*
 * Serving a decoder layer.  The calls below are the neighbours of the
 * quantized AllReduce in a served model: a key/value cache held with the same
 * int8 codes, and products with 4-bit weights.  They keep the conventions at
 * the top of this file (asynchronous, checked before anything is enqueued, no
 * allocation and no synchronization, capturable); what differs is said here.
 *
 * Microscaled 4-bit floating point ("mx4").  A block is QAR_MX4_BLOCK
 * consecutive elements of a row, the last block of a row padded with zeros:
 *
 *   scale  2^e  where 2^(e+2) <= absmax < 2^(e+3), e in -126 .. 125
 *               (subnormal blocks take e = -126, all-zero blocks e = -3);
 *               stored as the byte 127 + e
 *   code   the E2M1 value nearest to x_i / 2^e among 0, .5, 1, 1.5, 2, 3, 4, 6
 *          (codes 0 .. 7), ties to the even code, larger quotients become 6;
 *          bit 3 is the sign
 *   value  e2m1(code) * 2^e, exact in binary32 and in bf16
 *
 * Codes are uint8_t[rows][nb][16] with nb = ceil(cols / 32), the even element
 * in the low nibble; scales are uint8_t[rows][nb].  Scale bytes made elsewhere
 * may be 0 .. 254 (0 is 2^-127).  Elements must be finite, as everywhere: a NaN
 * or an infinity has no code, and its block's result is unspecified.
 */
#define QAR_MX4_BLOCK 32
#define QAR_MX4_MAX_DIM ((size_t)1 << 24) /* of rows and of columns */

/*
 *   x       [in]  rows * cols elements of `dtype`, 16-byte aligned.
 *   codes   [out] 16-byte aligned; scales [out].
 */
qar_status qar_mx4_quantize(const void* x, qar_dtype dtype, size_t rows, size_t cols, uint8_t* codes,
                            uint8_t* scales, void* stream);
/*
 *   out     [out] rows * cols elements of out_dtype, 16-byte aligned.
 */
qar_status qar_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, size_t rows, size_t cols, void* out,
                              qar_dtype out_dtype, void* stream);

/*
 * out[r][c] = sum over k of q(x)[r][k] * w[c][k]: the activations x are
 * quantized on the way (as qar_mx4_quantize does), the weights are mx4 rows
 * [cols][inner].  Products are exact, sums binary32, the result is rounded
 * once.  The order of a sum depends on the sizes alone, so equal calls give
 * equal bits.
 *   x, out     rows * inner elements of `dtype` and rows * cols of out_dtype,
 *              16-byte aligned.
 *   codes, scales  [in] the weights, codes 16-byte aligned.
 *   workspace  [scratch] qar_mx4_linear_workspace_bytes(rows, inner, cols)
 *              bytes, 256-byte aligned; NULL when that is 0 (few rows).  It
 *              needs no preparation and holds nothing between calls; calls
 *              that may run at the same time need one each.
 */
size_t qar_mx4_linear_workspace_bytes(size_t rows, size_t inner, size_t cols);
qar_status qar_mx4_linear(const void* x, qar_dtype dtype, size_t rows, size_t inner, const uint8_t* codes,
                          const uint8_t* scales, size_t cols, void* out, qar_dtype out_dtype, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * The same product with an epilogue:
 *   out[r][c] = residual[r][c] + activation(sum + bias[c])
 * where sum is the one above, all in binary32, the result rounded once.
 *   bias       [in, optional] cols elements of out_dtype, 16-byte aligned.
 *   activation  y -> y, max(y, 0), y / (1 + e^-y), y (1 + erf(y / sqrt 2)) / 2, or
 *              y (1 + tanh(sqrt(2 / pi) (y + 0.044715 y^3))) / 2; each to 2^-16
 *              of itself where the result is bf16, else to 2^-21 (below 2^-119
 *              it may be 0).  Of +infinity each is +infinity; of -infinity the
 *              second and fourth are 0, the third and fifth NaN.
 *   residual   [in, optional] rows * cols elements of out_dtype, 16-byte
 *              aligned; may be `out` itself.
 *   workspace  that of qar_mx4_linear.
 */
typedef enum qar_activation QAR_ENUM_BASE {
    QAR_ACT_NONE = 0,
    QAR_ACT_RELU = 1,
    QAR_ACT_SILU = 2,
    QAR_ACT_GELU = 3,
    QAR_ACT_GELU_TANH = 4
} qar_activation;

qar_status qar_mx4_linear_fused(const void* x, qar_dtype dtype, size_t rows, size_t inner, const uint8_t* codes,
                                const uint8_t* scales, size_t cols, const void* bias, qar_activation activation,
                                const void* residual, void* out, qar_dtype out_dtype, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * The paged cache of keys and values held in 8 bits ("kv8").  A pool of
 * `pages` pages of QAR_KV8_PAGE tokens; page p holds, for each of kv_heads
 * heads, the keys' int8 codes [token][dim], the values' [dim][token], and a
 * binary32 scale for either (codes, scales and values as for the int8 blocks
 * at the top of this file, the page of a head being the block).  Sequence b's
 * token t lies in page page_table[b][t / QAR_KV8_PAGE] at t % QAR_KV8_PAGE.
 * Codes behind a sequence's last token are unspecified.
 *   An entry of the page table outside 0 .. pages - 1 is a page that is not
 * there: nothing is written to it, its tokens read as zeros and attention
 * sees none of them.  Lengths below 0 count as 0 and those above
 * table_width * QAR_KV8_PAGE as that.  Pages may be shared by sequences that
 * only read them; a page that a call writes may appear once in its table.
 *   dim is 64, 128 or 256 (QAR_ERR_UNSUPPORTED otherwise); k and v are
 * 16-byte aligned, the other pointers 4-byte.
 */
#define QAR_KV8_PAGE 64

typedef struct qar_kv8_cache {
    int8_t* k;                 /* [pages][kv_heads][QAR_KV8_PAGE][dim] */
    float* k_scales;           /* [pages][kv_heads] */
    int8_t* v;                 /* [pages][kv_heads][dim][QAR_KV8_PAGE] */
    float* v_scales;           /* [pages][kv_heads] */
    const int32_t* page_table; /* [batch][table_width] */
    int32_t* lengths;          /* [batch]: tokens held */
    uint32_t pages, kv_heads, dim, batch, table_width;
} qar_kv8_cache;

/*
 * `tokens` new tokens of every sequence enter at positions starts[b] .. of
 * sequence b.  A page that they enter behind older tokens (positions below
 * starts[b]) keeps its scale unless they raise its absmax; then its older
 * values are quantized again with the new scale.  What the pages that they
 * enter held behind the last new token is lost: tokens are replaced from
 * starts[b] to the end, not in the middle.  `lengths` is neither read nor
 * written.  Positions behind the table and pages that are not there are
 * left out; a negative start leaves the sequence out.
 *   starts        [in] int32[batch].
 *   k_new, v_new  [in] [batch][tokens][kv_heads][dim] of `dtype`, 16-byte aligned.
 */
qar_status qar_kv8_append(const qar_kv8_cache* cache, const int32_t* starts, const void* k_new, const void* v_new,
                          qar_dtype dtype, uint32_t tokens, void* stream);

/*
 * Tokens starts[b] .. starts[b] + tokens - 1 of every sequence as values;
 * zeros behind its length (and everywhere for a negative start).
 *   k_out, v_out  [out] [batch][tokens][kv_heads][dim] of out_dtype, 16-byte aligned.
 */
qar_status qar_kv8_read(const qar_kv8_cache* cache, const int32_t* starts, uint32_t tokens, void* k_out,
                        void* v_out, qar_dtype out_dtype, void* stream);

/*
 * Causal attention of the last q_lens[b] tokens of every sequence over the
 * cache (which holds them already): query i of sequence b sees its first
 * lengths[b] - q_lens[b] + i + 1 tokens.
 *   out[b][i][j] = sum over t of p_t v_t,  p = softmax(scale * q . k_t)
 * with key head j / (heads / kv_heads) for query head j.  A row that sees no
 * token gives zeros, and so do rows i >= q_lens[b].  A NaN in a query makes
 * its row NaN and no other (and the weights of the tokens that the row sees).
 * Scores, maxima, sums and outputs are binary32; the softmax's numerators enter
 * the second product in binary16 (bf16 queries: each off by at most 2^-11 of
 * itself) or as two binary16 terms (binary32 queries: 2^-23).  Each enters times
 * its page's value scale over the largest value scale; below 2^-28 of the row's
 * largest numerator that product is off by up to 2^-39 of it instead.
 *   q, out     [batch][queries][heads][dim] of `dtype`, 16-byte aligned;
 *              heads % kv_heads == 0.
 *   q_lens     [in, optional] int32[batch]; NULL: `queries` for all.  Clipped
 *              to 0 .. queries.
 *   weights    [in/out, optional] float[batch][kv_heads][table_width * QAR_KV8_PAGE]:
 *              each token's p, summed over the queries and the heads that
 *              share its key head, is added.  No atomics: equal calls give
 *              equal bits.
 *   workspace  [scratch] qar_kv8_attention_workspace_bytes(...) bytes,
 *              256-byte aligned, as for qar_mx4_linear; with_weights says
 *              whether weights are passed.
 */
size_t qar_kv8_attention_workspace_bytes(uint32_t batch, uint32_t queries, uint32_t heads, uint32_t kv_heads,
                                         uint32_t dim, uint32_t table_width, qar_dtype dtype, int with_weights);
qar_status qar_kv8_attention(const qar_kv8_cache* cache, const void* q, qar_dtype dtype, uint32_t queries,
                             uint32_t heads, const int32_t* q_lens, float scale, float* weights, void* out,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same attention for a batch whose sequences share their first tokens:
 * group g is sequences starts[g] .. starts[g + 1] - 1, and its sequences' tables
 * name the same pages for their first prefix[g] tokens, as far as each has
 * tokens: one may be shorter, or have ended and hold none.  The pages wholly
 * among these are read once for all of the group's queries (through the table of
 * its first sequence, or of its longest one where the first is shorter), the
 * others sequence by sequence; the result is that of qar_kv8_attention up to the
 * order of the sums, whatever the lengths.
 * Sequences outside all groups share nothing.
 *   starts     [in] int32[groups + 1], ascending, 0 .. batch; 1 <= groups <= batch.
 *   prefix     [in] int32[groups]; below 0 counts as 0.
 *   workspace  [scratch] qar_kv8_attention_shared_workspace_bytes(...) bytes, as
 *              for qar_kv8_attention (never NULL).
 */
size_t qar_kv8_attention_shared_workspace_bytes(uint32_t batch, uint32_t queries, uint32_t heads, uint32_t kv_heads,
                                                uint32_t dim, uint32_t table_width, uint32_t groups);
qar_status qar_kv8_attention_shared(const qar_kv8_cache* cache, const void* q, qar_dtype dtype, uint32_t queries,
                                    uint32_t heads, const int32_t* starts, const int32_t* prefix, uint32_t groups,
                                    const int32_t* q_lens, float scale, void* out, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * Every sequence and head keeps `keep` tokens: its last min(recent, keep) and,
 * of the others, those with the largest weights, the lower position where
 * weights are equal (NaN counts as the largest).  A sequence of at most `keep`
 * tokens keeps all.  The kept tokens, in order, fill `into`'s pages from
 * position 0, each page quantized with its own scale, and into->lengths[b]
 * becomes min(lengths[b], keep).
 *   cache, into  equal batch, kv_heads and dim.  Their pages must be disjoint
 *                (one pool may hold both); tables and lengths are their own;
 *                into->table_width * QAR_KV8_PAGE >= keep.
 *   weights  [in]  float[batch][kv_heads][table_width * QAR_KV8_PAGE] (cache's),
 *                  16-byte aligned.
 *   kept     [out] int32[batch][kv_heads][keep]: the kept positions, ascending; -1 behind them.
 *   moved    [out] float[batch][kv_heads][keep]: their weights; 0 behind them.
 */
qar_status qar_kv8_evict(const qar_kv8_cache* cache, const qar_kv8_cache* into, const float* weights,
                         uint32_t recent, uint32_t keep, int32_t* kept, float* moved, void* stream);

/*
 * Head norms and rotary positions ("rotate").  The joint projection of a
 * layer's hidden states holds the queries of `heads` heads, then the keys and
 * then the values of kv_heads heads each.  Queries and keys are normed head by
 * head and rotated by their position, values are copied:
 *   y = x / sqrt(mean(x^2) + eps) * gain      (QAR_ROTATE_NORM; gain where one is passed)
 *   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * frequencies[j]
 * for pair j = 0 .. pairs - 1 of a head's channels: (j, j + pairs), or (2 j,
 * 2 j + 1) with QAR_ROTATE_NEIGHBOURS; channels from 2 * pairs on are not
 * rotated.  The angle is formed and reduced in 64 bits, the rest is binary32,
 * each result is rounded once.  A NaN or an overflowing sum of squares in a
 * head stays in that head.
 *   qkv        [in]  [batch][tokens][heads + 2 kv_heads][dim] of `dtype`, 16-byte aligned.
 *   positions  [in]  int32[batch], each sequence's first token's (the i-th has
 *                    i more), or int32[batch][tokens] with QAR_ROTATE_EACH_TOKEN.
 *   frequencies  [in]  float[pairs], radians a position; 0 <= pairs <= dim / 2 (NULL where 0).
 *   q_gain, k_gain  [in, optional]  [dim] of `dtype`, 16-byte aligned; only with QAR_ROTATE_NORM.
 *   q, k, v    [out] [batch][tokens][heads or kv_heads][dim] of `dtype`, 16-byte aligned.
 * dim is 64, 128 or 256; eps is finite and at least 0 (a head of zeros gives
 * zeros where it is more).
 */
#define QAR_ROTATE_NORM 1u
#define QAR_ROTATE_NEIGHBOURS 2u
#define QAR_ROTATE_EACH_TOKEN 4u

qar_status qar_norm_rotate(const void* qkv, qar_dtype dtype, size_t batch, size_t tokens, uint32_t heads,
                           uint32_t kv_heads, uint32_t dim, const int32_t* positions, const float* frequencies,
                           uint32_t pairs, const void* q_gain, const void* k_gain, float eps, uint32_t flags, void* q,
                           void* k, void* v, void* stream);

/*
 * Owners of the cache's pages.  refs[p] (int32[cache->pages], the caller's)
 * counts the entries of all page tables that name page p; a page whose count is
 * not above 0 is free.  Sequences may share the pages of tokens that they have
 * in common; a page is written only by a sequence that owns it alone.  All is
 * done on the device (nothing is read back, calls can be captured), and every
 * result is that of serving the sequences in order, so equal calls give equal
 * tables.  Entries outside the pool are pages that are not there, as everywhere.
 * Caches of several layers whose page tables are the same take one call for the
 * table, and one qar_kv8_copy for each layer.  batch < 2^24 and
 * batch * table_width < 2^31.
 *
 * fork: sequence b of `into` goes on from sequence parents[b] of `cache`: its
 * length, and the same pages up to it (their counts grow); no entries behind.
 * A parent outside 0 .. cache->batch - 1 gives an empty sequence.  The pool is
 * one (k, v and scales are not used); into's table and lengths are overwritten,
 * without anything being released.
 *   parents  [in] int32[into->batch].   into->table_width >= cache->table_width.
 */
qar_status qar_kv8_fork(const qar_kv8_cache* cache, int32_t* refs, const int32_t* parents, const qar_kv8_cache* into,
                        void* stream);
/*
 * free: every sequence is cut to its first min(lengths[b], max(keep[b], 0))
 * tokens (to none where keep is NULL).  Pages wholly behind them, those given
 * ahead among them, are released and their entries become -1.  keep may be
 * cache->lengths itself: then only what was given ahead is released.
 */
qar_status qar_kv8_free(const qar_kv8_cache* cache, int32_t* refs, const int32_t* keep, void* stream);
/*
 * reserve: pages for tokens[b] more tokens of every sequence.  Sequences are
 * served in order.  One that goes on in a partly filled page with other owners
 * gets a page in its place: source[b] and target[b] are then the two, whose
 * content the caller copies (qar_kv8_copy) before it appends; otherwise both
 * are -1.  Behind its last page every page up to lengths[b] + tokens[b] that is
 * not there is given; those that are there count as its own, so a sequence that
 * is to lose tokens is cut back with qar_kv8_free and not by its length alone.
 * Pages are taken lowest free number first.  When none is left a sequence keeps
 * what it got.  lengths are not changed.
 *   tokens   [in]  int32[batch]; below 1 counts as none.
 *   room     [out] int32[batch]: for how many tokens there is room now, at most
 *                  tokens[b]; 0 for one whose shared or missing page could not be
 *                  replaced (a partly filled page that is not there is not).
 *   source, target  [out] int32[batch].
 * batch <= QAR_KV8_MAX_SEQUENCES.
 */
#define QAR_KV8_MAX_SEQUENCES 4096
qar_status qar_kv8_reserve(const qar_kv8_cache* cache, int32_t* refs, const int32_t* tokens, int32_t* room,
                           int32_t* source, int32_t* target, void* stream);
/*
 * compact: with L pages in use, those from number L on change places with free
 * ones below L, the lowest with the lowest.  refs and the cache's table follow;
 * what other tables name is found in the lists.  The caller copies the pages
 * (qar_kv8_copy), and may then give the pool from page L on to others.
 *   source, target  [out] int32[pages / 2]: the moves, -1 behind them.  (A cache
 *                   without sequences is refused here: lists would be left unset.)
 */
qar_status qar_kv8_compact(const qar_kv8_cache* cache, int32_t* refs, int32_t* source, int32_t* target, void* stream);
/*
 * copy: page target[i] of `into` becomes page source[i] of `cache`, all heads,
 * keys and values with their scales, for every i whose two pages are there.  The
 * two may be one pool, or pools of equal kv_heads and dim.  A target may appear
 * once, and not as a source.  Tables and lengths are not used.
 */
qar_status qar_kv8_copy(const qar_kv8_cache* cache, const qar_kv8_cache* into, const int32_t* source,
                        const int32_t* target, uint32_t count, void* stream);

/* Static text for a status code. */
const char* qar_status_string(qar_status status);

/* Text of the last QAR_ERR_HIP raised on the calling thread ("" if none). */
const char* qar_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* QAR_H */
