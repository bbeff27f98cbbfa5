/*
 * nvfp4.h -- C ABI of the NVFP4 W4A4 small-M decode library for GB300 (sm_103a).
 *
 * What it computes (the ReSET pages):
 *   - NVFP4 = E2M1 4-bit elements, one E4M3 scale per 16 consecutive elements
 *     along K, one FP32 global scale per tensor (ReSET reading note, §2.1;
 *     §6.1 setup: "E2M1 elements, E4M3 block scales, group size 16").
 *   - The small-M decode projection Y = dequant(Xq) . dequant(Wq)^T for
 *     M = 1..8 active tokens, computed without a 128-row tensor-core tile
 *     (ReSET project page, "Why a CUDA-core NVFP4 kernel?" and "Core
 *     contribution -- the nvfp4r CUDA-core kernel", design choices C1-C3).
 *   - The ReSET step-aware temperature sampler: token entropy, online step
 *     entropy estimate (HSE), step-aware threshold (SAT), two-temperature
 *     sample (project page, "Step-aware temperature scaling"; reading note
 *     §3.1, §4.1-§4.3).
 *
 * Conventions for every entry point:
 *   - Data pointers are DEVICE pointers owned by the caller; the library keeps
 *     no reference after the call returns and allocates nothing.
 *   - Calls are asynchronous on `stream` (0 = the legacy default stream) and
 *     may be captured into a CUDA graph, except where a function says otherwise.
 *   - Argument errors are reported synchronously, before anything is launched:
 *     NVFP4_ERR_NULL, NVFP4_ERR_SHAPE, NVFP4_ERR_ALIGN, NVFP4_ERR_RANGE.
 *     A failed launch returns NVFP4_ERR_CUDA; nvfp4_last_cuda_error() names it.
 *   - Tensors are row-major and dense.  NVFP4 tensor layout:
 *       codes  uint8 [rows, K/2]  element 2j in the low nibble of byte j,
 *                                 element 2j+1 in the high nibble;
 *       scales uint8 [rows, K/16] E4M3 (OCP "fn") scale of elements 16b..16b+15,
 *                                 not interleaved;
 *       global float (one, on the device) -- dequant: x = e2m1(c) * e4m3(s) * global.
 *   - Calls on distinct streams are independent, except where a function
 *     says that concurrent calls share a buffer.
 */
#ifndef NVFP4_GB300_H
#define NVFP4_GB300_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum nvfp4_status {
  NVFP4_OK = 0,
  NVFP4_ERR_NULL = 1,   /* a required pointer is NULL */
  NVFP4_ERR_SHAPE = 2,  /* a size is negative, too large or not a required multiple */
  NVFP4_ERR_ALIGN = 3,  /* a pointer is not aligned as the function requires */
  NVFP4_ERR_RANGE = 4,  /* a parameter value is out of range (M, temperatures, w, ...) */
  NVFP4_ERR_CUDA = 5,   /* a CUDA runtime call or a kernel launch failed */
  NVFP4_ERR_DEVICE = 6  /* the current device is not a Blackwell sm_100-family GPU */
} nvfp4_status;

/* Static string for a status code. */
const char* nvfp4_status_str(nvfp4_status s);

/* Text of the last CUDA error seen by this library in the calling thread (static storage). */
const char* nvfp4_last_cuda_error(void);

/* Library ABI version: (major << 16) | minor. */
int nvfp4_version(void);

/*
 * Reads and clears the device error bits of the current device (the OR of
 * every error any kernel recorded since the last read).  A kernel sets a bit
 * when one of its bounded waits gave up, then returns early with incomplete
 * outputs:
 *   bit 0 (1)  a wait on an mbarrier (a TMA copy or an MMA that never completed);
 *   bit 1 (2)  reset_sample called with a state built for a smaller window;
 *   bit 2 (4)  a GEMV CTA's wait for another CTA's partial sum.  After this
 *              error the GEMV workspace may hold a partial sum published after
 *              the wait gave up: zero the workspace again before its next use;
 *   bit 3 (8)  a KV cache kernel met a slot or a page outside the cache, or a
 *              length or row range outside its table, and skipped it;
 *   bit 4 (16) reset_sample met a row that it can sample no token of;
 *   bit 5 (32) nvfp4_moe_route met a token whose logits give no choice;
 *   bit 6 (64) an expert kernel met an expert, offset, pair or place outside
 *              its tables and skipped it.
 * Synchronous (it copies a few bytes from the device); not for use inside
 * stream capture.
 */
nvfp4_status nvfp4_device_status(unsigned int* code);

/* ------------------------------------------------------------------------ */
/* Quantizer: BF16 -> NVFP4                                                   */
/* ------------------------------------------------------------------------ */
/*
 * Quantizes x[rows, K] (BF16 bit patterns) by the NVFP4 two-level recipe, all
 * in FP32 with IEEE rounding at each step:
 *   amax = max|x| over the whole tensor; global = amax / 2688 (448 * 6);
 *   per 16-element block: s = E4M3_rne_satfinite(max|x_block| / (6 * global));
 *   per element: code = E2M1_rne_satfinite(x / (e4m3(s) * global)).
 * The sign bit of each code is the sign bit of x (a negative value that rounds
 * to zero gives 0x8).  When e4m3(s) * global is 0 (all-zero block, a scale that
 * underflows, all-zero tensor) the code is the sign bit alone.
 * Format: ReSET reading note §2.1 and §6.1; the pages' activation quantizer
 * "Q" with a non-interleaved scale layout: reading note §5.3 (Table 3).
 *
 *   x_bf16   device, [rows, K] BF16, 16-byte aligned
 *   rows     >= 0 (activations: the M tokens; weights: N output channels)
 *   K        >= 0, multiple of 16
 *   codes    device, [rows, K/2], 16-byte aligned            (written)
 *   scales   device, [rows, K/16], 4-byte aligned            (written)
 *   global   device, one float, 4-byte aligned               (written)
 * Inputs with NaN or Inf are outside the contract (results unspecified).
 * rows == 0 or K == 0 writes global = 0.
 */
nvfp4_status nvfp4_quantize_act(const uint16_t* x_bf16, int rows, int K, uint8_t* codes,
                                uint8_t* scales, float* global_scale, cudaStream_t stream);

/*
 * Same recipe on FP32 input rows that are first rounded to BF16 (RNE): the
 * values quantized are exactly those nvfp4_quantize_act would see after a
 * FP32->BF16 cast.  Row r of the input starts at x + r * ld (ld >= K, in
 * floats), so a column slice [0, K) of a wider matrix can be quantized in
 * place (the decode step feeds the query columns of the qkv output to the o
 * projection this way).  x 16-byte aligned, ld a multiple of 4.
 */
nvfp4_status nvfp4_quantize_f32(const float* x, int rows, int K, int ld, uint8_t* codes,
                                uint8_t* scales, float* global_scale, cudaStream_t stream);

/*
 * SiLU(gate) * up on FP32 gate_up[rows, 2*I] (gate = columns [0, I), up =
 * columns [I, 2I)), each product computed in FP32 and rounded to BF16, then
 * quantized by the recipe above into codes[rows, I/2], scales[rows, I/16].
 * I a multiple of 16; gate_up 16-byte aligned.  (The MLP of the decode step
 * between the gate_up and down projections.)
 */
nvfp4_status nvfp4_silu_mul_quantize(const float* gate_up, int rows, int I, uint8_t* codes,
                                     uint8_t* scales, float* global_scale, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Small-M NVFP4 GEMV                                                         */
/* ------------------------------------------------------------------------ */
/*
 * y[m, n] = xg * wg * sum_k e2m1(xq[m,k]) e4m3(xs[m,k/16]) e2m1(wq[n,k]) e4m3(ws[n,k/16])
 * for m < M, n < N: the decode projection Y = X W^T of the ReSET project page
 * ("Core contribution": one CTA group reuses each streamed weight tile for all
 * M tokens, several accumulator chains per thread, register-only dequant).
 * Accumulation is FP32 across blocks; the result is within
 * 1e-3 * sum_k |x_k w_k| + 1e-6 of the exact product.
 *
 *   xq, xs, xg   activations in NVFP4 layout, [M, K/2], [M, K/16], one float
 *   M            1..8
 *   wq, ws, wg   weights in NVFP4 layout, [N, K/2], [N, K/16], one float
 *   N            1 .. 2^20
 *   K            >= 256, multiple of 256
 *   y            device, [M, N] FP32 (written)
 *   workspace    device scratch of at least nvfp4_gemv_workspace_bytes(M, N, K)
 *                bytes, 256-byte aligned, ZEROED ONCE before its first use
 *                (cudaMemset); every call leaves it ready for the next one,
 *                whatever the shape of the next call -- unless the call
 *                recorded device error bit 2 (nvfp4_device_status): zero it
 *                again then.
 *                Calls that overlap in time on the GPU must use different
 *                workspaces.
 * Co-residency: the kernel's CTAs (two per SM, one grid of up to 2 x the SM
 * count) exchange partial sums and wait for one another, so all of them must
 * be resident at once.  That holds when the call has the GPU to itself or
 * shares it with other kernels that finish; under MPS limits or green contexts
 * that cap the SMs a context may use, or beside a kernel that never ends, a
 * CTA's wait can run out: the call then records bit 2 and its y is wrong.
 * Alignment: xq, wq, xs, ws 16-byte aligned; y 16-byte aligned.
 */
size_t nvfp4_gemv_workspace_bytes(int M, int N, int K);

nvfp4_status nvfp4_gemv_smallm(const uint8_t* xq, const uint8_t* xs, const float* xg, int M,
                               const uint8_t* wq, const uint8_t* ws, const float* wg, int N, int K,
                               float* y, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * nvfp4_gemv_smallm computed by a second, independent kernel on the CUDA cores:
 * the pages' own design (ReSET project page, "Core contribution -- the nvfp4r
 * CUDA-core kernel": each weight tile streamed once for all M tokens (C1),
 * several FP32 accumulator chains per thread (C2), dequantization in
 * registers (C3)), with each 16-element block summed exactly in integers.
 * Same arguments, result tolerance, workspace and errors as
 * nvfp4_gemv_smallm; not the fast path (the tensor-core kernel is), kept so
 * that two implementations can be checked against each other.
 */
nvfp4_status nvfp4_gemv_smallm_cudacore(const uint8_t* xq, const uint8_t* xs, const float* xg, int M,
                                        const uint8_t* wq, const uint8_t* ws, const float* wg, int N, int K,
                                        float* y, void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream);

/*
 * Test hook for the tensor-core GEMV's bounded wait (no counterpart in the
 * pages).  For every later tensor-core GEMV launch in the process:
 * flag_spin_limit = how many times a CTA polls another CTA's partial sum
 * before giving up (0 = the default, about 2^24 polls), and drop_records != 0
 * makes every CTA skip publishing its partial sums, so that the CTA finishing
 * a split tile waits until the limit, records device error bit 2 and writes a
 * wrong y.  Lets a test make the wait run out without any fault or hang.
 * Call nvfp4_test_gemv_fault(0, 0) to return to normal operation; not
 * thread-safe against concurrent GEMV calls.
 */
void nvfp4_test_gemv_fault(unsigned int flag_spin_limit, int drop_records);

/*
 * Packed weights.  The pages quantize the weights offline, from the BF16
 * checkpoint (ReSET reading note §6.1), and leave their memory layout to the
 * kernel.  nvfp4_pack_weights rewrites wq/ws into blocks of
 * 18432 bytes, one per [128-row tile t] x [256-K chunk c], stored in the order
 * (t, c) with c fastest, so that a GEMV streams each tile chunk as one
 * contiguous read:
 *   bytes [0, 16384)      codes of rows 128t .. 128t+127, K-bytes [128c, 128c+128):
 *                         the 16-byte piece j (0..7) of tile row r (0..127) at
 *                         r*128 + ((j XOR (r mod 8)) * 16)
 *   bytes [16384, 18432)  scales of those rows for blocks [16c, 16c+16): tile
 *                         row r at 16384 + 16 r
 * Rows n >= N of the last tile are zero.  The packed image holds the same
 * bytes as wq and ws (plus the zero rows); nothing is recomputed.
 *
 * nvfp4_packed_weight_bytes(N, K) = ceil(N/128) * (K/256) * 18432, or 0 for an
 * invalid shape (N 1 .. 2^20, K a positive multiple of 256).
 * nvfp4_pack_weights: wq [N, K/2], ws [N, K/16], packed (written) of at least
 * nvfp4_packed_weight_bytes bytes, all device, 16-byte aligned; asynchronous on
 * `stream`; wq/ws must not overlap `packed`.
 * nvfp4_gemv_smallm_packed: nvfp4_gemv_smallm with the weights given packed;
 * same result bits for the same inputs on the tensor-core path, same
 * workspace contract.
 */
size_t nvfp4_packed_weight_bytes(int N, int K);

nvfp4_status nvfp4_pack_weights(const uint8_t* wq, const uint8_t* ws, int N, int K, uint8_t* packed,
                                size_t packed_bytes, cudaStream_t stream);

nvfp4_status nvfp4_gemv_smallm_packed(const uint8_t* xq, const uint8_t* xs, const float* xg, int M,
                                      const uint8_t* wpacked, const float* wg, int N, int K, float* y,
                                      void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * nvfp4_quantize_act of a BF16 activation followed by nvfp4_gemv_smallm_packed,
 * as one call: y[m, n] = xg * wg * sum_k e2m1(xq[m,k]) e4m3(xs[m,k/16])
 * e2m1(wq[n,k]) e4m3(ws[n,k/16]), where wq, ws are the codes and scales the
 * packed image holds and xq, xs, xg exactly what nvfp4_quantize_act(x) would
 * write (the
 * activation quantizer "Q" in front of every decode projection: ReSET
 * reading note §5.3, Table 3).  y holds the same bits as the two calls.
 * For M <= 3 and M * K <= 65536 it is one launch (tuning knobs
 * NVFP4_QGEMV_MAX_M, NVFP4_QGEMV_MAX_MK): every CTA of the GEMV reads the
 * whole activation for its maximum and quantizes the 256-K chunks it
 * multiplies into shared memory, so the quantized activation never goes
 * through HBM and one kernel boundary of a decode chain disappears.  Larger
 * activations, or a CTA that would hold more than 24 chunks or quantize more
 * than 1024 blocks (NVFP4_QGEMV_MAX_BLOCKS), take two launches: the library
 * quantizes into the workspace, then multiplies.
 *   x        device, BF16 [M, K] row-major, 16-byte aligned
 *   M        1..8 (else NVFP4_ERR_RANGE)
 *   wpacked, wg, N, K   as nvfp4_gemv_smallm_packed
 *   y        device, [M, N] FP32, 16-byte aligned (written)
 *   xg_out   device float receiving the activation's global scale amax / 2688,
 *            4-byte aligned, or NULL
 *   workspace  device scratch of at least
 *            nvfp4_quantize_gemv_workspace_bytes(M, N, K) bytes, 256-byte
 *            aligned; the same contract as the GEMV workspace (zeroed once,
 *            left ready, one per set of calls that overlap on the GPU); a
 *            zeroed workspace may serve this call and the GEMV calls alike.
 * Errors, co-residency and device error bits as nvfp4_gemv_smallm.
 */
size_t nvfp4_quantize_gemv_workspace_bytes(int M, int N, int K);

/*
 * How nvfp4_quantize_gemv_packed runs a shape on the current device: 1 (one
 * launch), 2 (the quantizer, then the GEMV), 0 for a shape it rejects, -1
 * when the device cannot be queried.  No launch, no synchronization.
 */
int nvfp4_quantize_gemv_launches(int M, int N, int K);

nvfp4_status nvfp4_quantize_gemv_packed(const uint16_t* x_bf16, int M, const uint8_t* wpacked,
                                        const float* wg, int N, int K, float* y, float* xg_out,
                                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Prefill-sized NVFP4 GEMM (M up to 128)                                      */
/* ------------------------------------------------------------------------ */
/*
 * y[m, n] = xg * wg * sum_k e2m1(xq[m,k]) e4m3(xs[m,k/16]) e2m1(w[n,k]) e4m3(sw[n,k/16])
 * for m < M <= 128 and packed weights: the same product as
 * nvfp4_gemv_smallm_packed for a prefill-sized batch of tokens (the pages'
 * own tensor-core GEMM at M = 128: ReSET reading note §7.3, Table 16).  One
 * tcgen05 MMA covers 128 weight rows x 128 tokens x 64 K; each weight block is
 * read from HBM once per call.  FP32 accumulation: within
 * 1e-3 * sum_k |x_k w_k| + 1e-6 of the exact product.
 *   xq, xs, xg   activations, NVFP4 layout [M, K/2], [M, K/16] (16-byte
 *                aligned), one float
 *   M            1..128 (else NVFP4_ERR_RANGE)
 *   wpacked, wg  the weight in the nvfp4_pack_weights layout, one float
 *   N, K         N 1 .. 2^20, K a positive multiple of 256
 *   y            [M, N] FP32, 16-byte aligned (written)
 *   workspace    device scratch of at least nvfp4_gemm_workspace_bytes(M, N, K)
 *                bytes (a fixed size per device: 64 KB per SM), 256-byte
 *                aligned, ZEROED ONCE before its first use and left ready for
 *                the next call of any shape; zero it again after device error
 *                bit 2.  Calls that overlap on the GPU need different workspaces.
 * Co-residency and errors as nvfp4_gemv_smallm.  One CTA per SM.
 */
size_t nvfp4_gemm_workspace_bytes(int M, int N, int K);

nvfp4_status nvfp4_gemm_packed(const uint8_t* xq, const uint8_t* xs, const float* xg, int M,
                               const uint8_t* wpacked, const float* wg, int N, int K, float* y,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* BF16 GEMV (the decode step's lm_head)                                       */
/* ------------------------------------------------------------------------ */
/*
 * y[m, n] = sum_k x[m, k] * w[n, k], BF16 inputs, FP32 accumulation and output.
 * M 1..8, K a multiple of 8 with M * K <= 51200 (x is held in shared memory as
 * FP32), all pointers 16-byte aligned.  Larger M * K returns NVFP4_ERR_SHAPE.
 */
nvfp4_status nvfp4_bf16_gemv(const uint16_t* x, int M, const uint16_t* w, int N, int K, float* y,
                             cudaStream_t stream);

/*
 * The same BF16 GEMV on the tensor cores (tcgen05 kind::f16, BF16 x BF16 ->
 * FP32 accumulator in TMEM), on the NVFP4 GEMV's kernel: weight tiles of
 * [128 rows x 64 K] streamed through a shared-memory ring by TMA, Stream-K
 * split over the tiles' K chunks, the same deterministic fix-up.  It needs
 * the records region of a GEMV workspace:
 *   nvfp4_bf16_gemv_workspace_bytes(M, N, K): bytes of workspace needed (0 for
 *   an invalid shape); any buffer that satisfies nvfp4_gemv_workspace_bytes
 *   for the same M also satisfies it, so one zeroed workspace serves both.
 *   x [M, K], w [N, K] BF16 row-major, y [M, N] FP32, all device, 16-byte
 *   aligned; M 1..8, N 1 .. 2^20, K a positive multiple of 64; workspace
 *   256-byte aligned, ZEROED ONCE before its first use, left ready for the
 *   next call.  FP32 accumulation: within 1e-4 * sum_k |x_k w_k| + 1e-6 of
 *   the exact product.  Errors as nvfp4_gemv_smallm.
 */
size_t nvfp4_bf16_gemv_workspace_bytes(int M, int N, int K);

nvfp4_status nvfp4_bf16_gemv_tc(const uint16_t* x, int M, const uint16_t* w, int N, int K, float* y,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * RMS normalization of FP32 rows to BF16 (no gain):
 *   out[r, k] = BF16( x[r, k] / sqrt( (1/K) sum_k x[r, k]^2 + eps ) )
 * Row r of the input starts at x + r * ld (ld >= K, in floats); out is
 * [rows, K] row-major.  The sum of squares is FP32 (in a fixed order per K),
 * the square root and the division IEEE; results are within one BF16 rounding
 * of the exact value.  K a multiple of 4, ld a multiple of 4, x 16-byte and
 * out 8-byte aligned, eps >= 0.
 * The pages' decode step runs inside a Qwen3 decoder, whose layers normalize
 * their inputs (ReSET reading note §6.1: Qwen3 models); the synthetic decode
 * step puts this in front of the qkv and gate_up projections so that a chain
 * of many layers keeps its magnitude (SiLU(gate)*up squares it otherwise).
 */
nvfp4_status nvfp4_rms_norm_bf16(const float* x, int rows, int K, int ld, float eps, uint16_t* out,
                                 cudaStream_t stream);

/*
 * nvfp4_rms_norm_bf16 followed by nvfp4_quantize_act, in one launch: the BF16
 * rows r = BF16(x / sqrt((1/K) sum x^2 + eps)) are quantized by the recipe of
 * nvfp4_quantize_act (one global scale over all rows) into codes [rows, K/2],
 * scales [rows, K/16] and global_scale.  The decode step's normalization in
 * front of the qkv and gate_up projections (see nvfp4_rms_norm_bf16).
 * The row's sum of squares is FP32 in a fixed order (it may differ from
 * nvfp4_rms_norm_bf16's order, so r may differ from that function's output by
 * one BF16 rounding where the exact value is that close to a boundary); the
 * codes are exactly nvfp4_quantize_act of r.  r_out, if not null, receives r
 * ([rows, K] BF16, 16-byte aligned).
 *   rows     0..8 (one CTA per row, the rows forming one thread-block cluster)
 *   K        16..16384, multiple of 16;  ld >= K, multiple of 4 (floats)
 *   eps      >= 0 (a zero row needs eps > 0)
 *   x        device FP32, row r at x + r * ld, 16-byte aligned
 *   codes    16-byte aligned; scales, global_scale 4-byte aligned (written)
 * Errors: NVFP4_ERR_SHAPE (K, ld), NVFP4_ERR_RANGE (rows > 8, eps < 0 or NaN),
 * NVFP4_ERR_NULL, NVFP4_ERR_ALIGN, NVFP4_ERR_CUDA (launch).  rows == 0 writes
 * global_scale = 0.
 */
nvfp4_status nvfp4_rms_norm_quantize(const float* x, int rows, int K, int ld, float eps, uint8_t* codes,
                                     uint8_t* scales, float* global_scale, uint16_t* r_out,
                                     cudaStream_t stream);

/* FP32 -> BF16 (RNE) elementwise cast of n values; x, y 16-byte aligned, n a multiple of 8. */
nvfp4_status nvfp4_f32_to_bf16(const float* x, size_t n, uint16_t* y, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Paged KV cache in NVFP4                                                     */
/* ------------------------------------------------------------------------ */
/*
 * K and V rows of D = head_dim elements (64 or 128) quantized to NVFP4 along D
 * (one E4M3 scale per 16 elements, one FP32 global scale for all of K and one
 * for all of V: x = e2m1(code) * e4m3(scale) * global), 9/16 byte an element.
 * The ReSET pages keep the KV cache in BF16 (reading note §6.1) and describe
 * no cache kernel; this part has no counterpart there.
 *
 * The cache is num_pages pages of page_size tokens (a multiple of 16).  Slot
 * s is token s % page_size of page s / page_size.  Memory: page, then kv
 * head, then groups of 16 tokens of 18 D bytes each:
 *   K codes  [pos][D/2 bytes]           pos = 8 (t/2 % 2) + 2 (t/4) + t % 2 for token t of the group
 *   K scales [r 8][c 4][i 2][D/64]      pos = 8 i + r, block of 16 elements = c D/64 + last index
 *   V codes  D = 128: [4][i 2][2][c 4][t0 2][8 bytes]  t = 4 c + 2 i + t0, elements 16 r .. 16 r + 15
 *                                       with r = 2 (first index) + (third index)
 *            D = 64:  [r 8][t 16][4 bytes]             elements 8 r .. 8 r + 7
 *   V scales [block][t]
 * of 8 D, D, 8 D and D bytes.  The even element of a pair sits in the low
 * nibble.  The order is that of the attention kernel's matrix fragments: each
 * of its threads finds what it multiplies in a few 16-byte pieces.
 */
typedef struct nvfp4_kv_cache {
  uint8_t* pages;         /* device, num_pages * nvfp4_kv_page_bytes bytes, 16-byte aligned */
  const float* k_global;  /* device, one float > 0                                         */
  const float* v_global;  /* device, one float > 0                                         */
  int num_pages;          /* >= 1; num_pages * page_size < 2^31                            */
  int page_size;          /* a multiple of 16, 16 .. 1024                                  */
  int kv_heads;           /* 1 .. 1024                                                     */
  int head_dim;           /* 64 or 128                                                     */
} nvfp4_kv_cache;

/* Element types of the rows that the functions below read. */
enum { NVFP4_DTYPE_F32 = 0, NVFP4_DTYPE_BF16 = 1 };

/* Bytes of one page (all kv heads), or 0 for an invalid shape. */
size_t nvfp4_kv_page_bytes(int page_size, int kv_heads, int head_dim);

/*
 * Gives the pages of ended requests back to the stack of free pages: for each
 * request b with ended[b] != 0, in order, its first ceil(lens[b] / page_size)
 * table entries are pushed, and free_count_out = free_count + their number.
 * The table is left as it is: the caller sets the request's length to 0.
 *   lens         device, [batch] int32, tokens held (negative counts as 0)
 *   ended        device, [batch] uint8
 *   batch        >= 0;  page_size a multiple of 16, 16 .. 1024
 *   block_table  device, [batch, table_width] int32 page ids
 *   free_pages   device, [free_capacity] int32, entries [0, free_count) are free pages (written behind them);
 *                pages beyond free_capacity are dropped
 *   free_count, free_count_out   device, one int32 each; may be the same address
 */
nvfp4_status nvfp4_kv_release(const int32_t* lens, const uint8_t* ended, int batch, int page_size,
                              const int32_t* block_table, int table_width, int32_t* free_pages, int free_capacity,
                              const int32_t* free_count, int32_t* free_count_out, cudaStream_t stream);

/*
 * Page table and slot map of a step from the requests' lengths.  Request b
 * holds ctx_lens[b] tokens and gets new_lens[b] more; the new tokens of all
 * requests are packed one request after the other.  With pages(n) =
 * ceil(n / page_size), it needs pages(ctx + new) - pages(ctx) new pages, taken
 * from the top of the free stack in request order, and
 *   block_table[b, pages(ctx) ..]  the new pages (other entries are kept);
 *   slots[i]      slot of new token i = block_table[b, pos / page_size] * page_size + pos % page_size;
 *   positions[i]  pos, its place in its request (ctx[b] for the first new token);
 *   cu_q[b]       first new token of request b; cu_q[batch] = their number;
 *   kv_lens[b]    ctx + new;
 *   free_count_out  pages left on the stack.
 * A request is refused when it needs pages and the needs of the requests up
 * to and including it exceed free_count, when pages(ctx + new) > table_width
 * or when a length is negative: it takes no page, its tokens' slots are -1 and
 * its kv_lens is its ctx (0 if negative).  A request that is invalid by its
 * lengths or its table counts as needing nothing; a negative new length counts
 * as no token.  Entries of slots and positions past the last token are -1 and 0.
 *   batch >= 1; max_tokens >= 0: entries of slots and positions; tokens beyond are not written
 *   info  device, two int32: requests refused, tokens planned (cu_q[batch])
 *   free_count_out may be free_count and kv_lens may be ctx_lens; outputs that overlap anything else are refused
 *   (NVFP4_ERR_SHAPE)
 */
nvfp4_status nvfp4_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int batch, int page_size,
                           int32_t* block_table, int table_width, const int32_t* free_pages, int free_capacity,
                           const int32_t* free_count, int32_t* free_count_out, int32_t* kv_lens, int32_t* cu_q,
                           int32_t* slots, int32_t* positions, int max_tokens, int32_t* info, cudaStream_t stream);

/*
 * Quantizes K and V rows into the cache: row i, head h at k + i * k_token_stride
 * + h * k_head_stride (strides in elements, the D elements of a row adjacent)
 * goes to slot slots[i] by the recipe of nvfp4_quantize_act with the cache's
 * global scales: s = E4M3(max|x_block| / (6 * global)), code = E2M1(x /
 * (e4m3(s) * global)).  FP32 rows are first rounded to BF16 (RNE).
 * A slot of -1 skips its row (padding); a slot outside the cache skips it and
 * records device error bit 3.  No two rows of a call may have the same slot
 * (their bytes would mix).
 *   k, v     device, 16-byte aligned, strides multiples of 16 bytes (any where there is one token, or one head)
 *   dtype    NVFP4_DTYPE_*;  tokens >= 0
 */
nvfp4_status nvfp4_kv_append(const void* k, const void* v, int dtype, int tokens, int64_t k_token_stride,
                             int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                             const int32_t* slots, const nvfp4_kv_cache* cache, cudaStream_t stream);

/*
 * nvfp4_kv_append with the rotation of positions on the way: q and k rows are rotated, q goes to q_out (BF16), k and v to
 * their slots.  With (c, s) = table[positions[i], m], pair m (m < rotated / 2) of a row turns from (a, b) to
 *   (a c - b s, b c + a s)          every product and sum rounded to FP32, the results to BF16 (RNE)
 * where (a, b) are elements (m, m + rotated/2) with NVFP4_ROPE_HALVES and (2m, 2m + 1) with NVFP4_ROPE_PAIRS; elements from
 * `rotated` on are rounded to BF16 alone.  K rows are quantized from their BF16 values by the recipe of nvfp4_kv_append.
 * FP32 rows are not rounded before they are rotated; v rows are first rounded to BF16.
 * A slot of -1 skips its row (padding: nothing of it is read, its q_out is zero).  So does, recording device error bit 3,
 * a slot outside the cache or a position outside the table.  No two rows of a call may have the same slot.
 *   q           device, [tokens, heads, head_dim] at q + i * q_token_stride + h * q_head_stride; heads 0 .. 65536
 *               (0: k and v alone; q and q_out are not looked at)
 *   k, v        as in nvfp4_kv_append;  dtype of all three;  all 16-byte aligned, strides multiples of 16 bytes
 *   positions   device, [tokens] int32
 *   table       device, [max_positions, rotated / 2, 2] FP32: cosine and sine, 16-byte aligned
 *   rotated     a multiple of 32, 32 .. head_dim
 *   q_out       device, [tokens, heads, head_dim] BF16, 16-byte aligned (written); not q, k or v
 */
enum { NVFP4_ROPE_HALVES = 0, NVFP4_ROPE_PAIRS = 1 };

nvfp4_status nvfp4_kv_append_rope(const void* q, const void* k, const void* v, int dtype, int tokens, int heads,
                                  int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                                  int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                                  const int32_t* positions, const float* table, int max_positions, int rotated, int style,
                                  const int32_t* slots, const nvfp4_kv_cache* cache, uint16_t* q_out, cudaStream_t stream);

/*
 * Reads rows back: k_out, v_out [tokens, kv_heads, head_dim] BF16 (16-byte
 * aligned) receive BF16(e2m1(code) * (e4m3(scale) * global)) of the slots'
 * rows, products in FP32; a slot of -1 gives zeros, one outside the cache gives zeros and
 * records device error bit 3.
 */
nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, const int32_t* slots, int tokens, uint16_t* k_out,
                           uint16_t* v_out, cudaStream_t stream);

/*
 * Attention of the packed query rows over the cache, causal from the bottom
 * right: query row i of request b (rows cu_q[b] .. cu_q[b+1]) stands at
 * position p = kv_lens[b] - (cu_q[b+1] - cu_q[b]) + i and sees the keys
 * j <= p, with window > 0 only those with j > p - window.  Query head h reads
 * kv head h / (heads / kv_heads):
 *   out[r, h, :] = sum_j softmax_j(scale * q[r, h] . K[j]) V[j]      (BF16)
 *   lse[r, h]    = log sum_j exp(scale * q[r, h] . K[j])             (FP32, natural log)
 * A row that sees no key gives out = 0, lse = -inf; so does one all of whose scores are -inf.  A row with a NaN
 * score, or one of +inf, gives NaN.
 * Precision: the keys' and values' dequantized values are exact.  FP32 queries are first rounded to BF16 (RNE); a
 * query enters the products as FP16 of q / 2^e, 2^e the power of two at its row's maximum (exact down to 2^-14 of
 * it).  Scores, their maxima, the sums and the accumulators are FP32.  The weights that multiply V are rounded to
 * FP16 (2^-11 of each, and those under 2^-25 of the maximum in use become 0), the weights that are summed are not.
 * The kernel for many rows moves its maximum only when a score exceeds it by a factor of 2^13, so its largest weight
 * need not be 1.  The result is rounded to BF16.
 *   q            device, [tokens, heads, head_dim] at q + r * q_token_stride + h * q_head_stride
 *                (elements; 16-byte aligned, strides multiples of 16 bytes, as of k and v above)
 *   heads        a multiple of kv_heads, at most 64 times it
 *   block_table  device, [batch, table_width] int32: page of tokens j * page_size ..
 *                Only entries of pages that some row sees are read; a page outside the cache is
 *                skipped (its keys count as unseen) and records device error bit 3, and so does a
 *                kv_lens beyond table_width * page_size (cut there) or a row range outside [0, tokens).  Where
 *                cu_q falls and ranges overlap, the call may compute nothing.
 *   kv_lens      device, [batch] int32
 *   cu_q         device, [batch + 1] int32, or NULL: one row a request (tokens == batch)
 *   max_q        >= 1: most rows of a request, as far as the caller knows (it chooses the kernel,
 *                not the result)
 *   out          device, [tokens, heads, head_dim] BF16, 16-byte aligned (written; rows of no request are left)
 *   lse          device, [tokens, heads] FP32, or NULL
 *   workspace    device scratch of nvfp4_kv_attention_workspace_bytes bytes, 256-byte aligned, its first
 *                4096 bytes ZEROED ONCE before its first use; every call leaves it ready for the next one of
 *                any shape that fits.  Calls that overlap on the GPU need different workspaces.
 */
size_t nvfp4_kv_attention_workspace_bytes(int batch, int tokens, int heads, int kv_heads, int head_dim);

nvfp4_status nvfp4_kv_attention(const void* q, int dtype, int tokens, int64_t q_token_stride, int64_t q_head_stride,
                                int heads, const nvfp4_kv_cache* cache, const int32_t* block_table, int table_width,
                                const int32_t* kv_lens, const int32_t* cu_q, int batch, int max_q, float scale,
                                int window, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Experts: routing, and the chosen experts' NVFP4 products                    */
/* ------------------------------------------------------------------------ */
/*
 * A layer with experts sends each token to top_k of them.  A PAIR is a token t
 * and its j-th expert, number t * top_k + j.  A PLAN of the pairs is
 *   offsets  [experts + 1]        the pairs of expert e stand at places
 *                                 offsets[e] .. offsets[e+1];
 *   pairs    [tokens * top_k]     the pair at each place, those of an expert
 *                                 in the order of their numbers; -1 behind
 *                                 offsets[experts];
 *   places   [tokens * top_k]     the place of each pair, -1: it has none.
 * The ReSET pages describe dense layers only; this part has no counterpart
 * there.  experts 1 .. 512, top_k 1 .. 32, tokens * top_k < 2^31.
 * The activations' global scale is one for all experts, as nvfp4_quantize_act
 * gives it: experts calibrated with an input scale each are not covered.
 * Workspaces keep no state; calls that overlap on the GPU need different ones.
 */
enum { NVFP4_MOE_SOFTMAX = 0, NVFP4_MOE_SIGMOID = 1 };

typedef struct nvfp4_moe_router {
  int top_k;        /* experts of a token, 1 .. 32                                            */
  int score;        /* NVFP4_MOE_*: softmax over all experts, or a sigmoid of each            */
  int groups;       /* experts e / (experts / groups) form a group; 1 .. 32, divides experts  */
  int top_groups;   /* groups a token may choose from, 1 .. groups                            */
  int group_best;   /* 1 or 2: a group's rank is by the sum of its so many largest values     */
  int renormalize;  /* non-zero: the weights of a token's experts are divided by their sum    */
  float scale;      /* and multiplied by this, finite                                         */
} nvfp4_moe_router;

/* Scratch of nvfp4_moe_route and nvfp4_moe_plan; 0 for calls that need none.  No state: nothing is kept in it. */
size_t nvfp4_moe_route_workspace_bytes(int tokens, int experts);

/*
 * Scores, choice, weights and plan from router logits x[t, e]:
 *   s[t, e] = softmax_e(x[t, :]) or 1 / (1 + exp(-x[t, e]))
 *   v[t, e] = s[t, e] + bias[e]          (what the choice goes by; without a bias the order of x)
 *   with top_groups < groups: the top_groups groups with the largest sums of their group_best largest v stay
 *   ids[t, :]     = the top_k experts with the largest v, in that order
 *   weights[t, j] = s[t, ids[t, j]], divided by the row's sum if renormalize, times scale          (FP32)
 * Equal values go to the lowest expert (or group).  Values are told apart as 64-bit arithmetic tells them: where FP32
 * cannot settle the order, the token is chosen again in FP64.  Renormalized weights do not underflow with their sum.
 * A token with a NaN among its logits (or biases), and with softmax one with a logit of +inf or with -inf alone, gives
 * no choice: ids -1, weights 0, no pair; device error bit 5 is recorded.  Logits of -inf are experts of score 0.
 *   logits   device, [tokens, experts] of dtype NVFP4_DTYPE_*, row t at logits + t * ld (elements)
 *   bias     device, [experts] FP32, or NULL
 *   rows     device, [tokens] uint8, or NULL: tokens with rows[t] == 0 are not read and get ids -1, weights 0, no pair
 *   ids, weights   device, [tokens, top_k] int32 / FP32 (written)
 *   offsets, pairs, places   the plan (written)
 *   workspace      device scratch, 4-byte aligned; may be NULL where the size is 0
 */
nvfp4_status nvfp4_moe_route(const void* logits, int dtype, int tokens, int experts, int64_t ld,
                             const nvfp4_moe_router* router, const float* bias, const uint8_t* rows, int32_t* ids,
                             float* weights, int32_t* offsets, int32_t* pairs, int32_t* places, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/*
 * The plan of a choice made elsewhere: ids [tokens, top_k] int32, -1 for no expert; ids outside [0, experts) are no
 * pair either and record device error bit 6.  An expert may stand twice in a row.
 */
nvfp4_status nvfp4_moe_plan(const int32_t* ids, int tokens, int top_k, int experts, int32_t* offsets, int32_t* pairs,
                            int32_t* places, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Packed expert weights.  nvfp4_moe_pack_weights rewrites the row-major NVFP4 matrices of all experts, wq
 * [experts, N, K/2] and ws [experts, N, K/16], into blocks of 18432 bytes, one per (expert, tile of 128 rows, 256 of K),
 * in this order, K fastest:
 *   bytes [0, 16384)      the 16-byte piece j (0..7) of the codes of tile row r at r*128 + ((j XOR (r mod 8)) * 16)
 *   bytes [16384, 18432)  scales of 16-element blocks 4q .. 4q+3 (q 0..3) of tile row r at
 *                         16384 + q*512 + (r mod 32)*16 + (r/32)*4
 * With gated != 0 the matrix is gate and up, N = 2 I, gate rows [0, I), up rows [I, 2I), I a multiple of 64, and their
 * rows alternate in the tiles: row 2i is gate row i, row 2i+1 up row i.  Rows beyond N and elements beyond K are zero.
 *   nvfp4_moe_packed_weight_bytes = experts * ceil(N/128) * ceil(K/256) * 18432, or 0 for an invalid shape:
 *   experts 1 .. 512, N 1 .. 2^20, K a multiple of 64, 64 .. 2^20
 *   wq, packed 16-byte aligned, ws 4-byte aligned; packed must not overlap wq or ws
 */
size_t nvfp4_moe_packed_weight_bytes(int experts, int N, int K, int gated);

nvfp4_status nvfp4_moe_pack_weights(const uint8_t* wq, const uint8_t* ws, int experts, int N, int K, int gated,
                                    uint8_t* packed, size_t packed_bytes, cudaStream_t stream);

/*
 * Gate and up products of the chosen experts, and SiLU(gate) * up, in one pass over their weights: with pair p at place q
 * (p = pairs[q]), token t = p / top_k and expert e (offsets[e] <= q < offsets[e+1]),
 *   g = xg wg[e] sum_k x[t, k] w[e, i, k],  u = the same with w[e, inter + i, k]       (FP32)
 *   h[q, i] = BF16(g / (1 + exp(-g)) * u)          (0 for g below -88.72, where FP32's exp(-g) overflows)
 * Rows of h behind offsets[experts] are zero, so that nvfp4_quantize_act may take all of h.
 *   xq, xs, xg   activations in NVFP4 layout, [tokens, K/2] 16-byte, [tokens, K/16] 4-byte aligned, one float
 *   wpacked, wg  packed with gated != 0 (N = 2 inter), 16-byte aligned; [experts] FP32 global scales
 *   inter        a multiple of 64;  K a multiple of 64
 *   h            device, [tokens * top_k, inter] BF16, 16-byte aligned (written)
 *   workspace    device scratch of nvfp4_moe_gate_up_workspace_bytes bytes (0 for few tokens, or few pairs an expert),
 *                256-byte aligned; no state
 * Only the weights of experts that have pairs are read.  Sums of a product are FP32 in an order that the shape and the
 * plan fix: the same inputs give the same bits.  Pairs and places outside their tables are taken into them or skipped and
 * record device error bit 6 (the rows concerned mean nothing), as do offsets that do not begin at 0, fall or lie outside
 * [0, tokens * top_k]: a plan of such is one without pairs.
 */
size_t nvfp4_moe_gate_up_workspace_bytes(int tokens, int top_k, int experts, int K);

nvfp4_status nvfp4_moe_gate_up(const uint8_t* xq, const uint8_t* xs, const float* xg, int tokens, int top_k,
                               const int32_t* offsets, const int32_t* pairs, const uint8_t* wpacked, const float* wg,
                               int experts, int inter, int K, uint16_t* h, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * Down products of the chosen experts, summed over a token's experts:
 *   y[t, n] = sum_j weights[t, j] hg wg[e] sum_k h[place(t, j), k] w[e, n, k]          (FP32)
 * over the pairs of t that have a place (none: 0).  No product is rounded on the way.  Up to 64 tokens the pairs are gone by,
 * beyond them the places: one outside [0, offsets[experts]) has no product, is skipped and records device error bit 6.
 *   hq, hs, hg   NVFP4 rows by place, [tokens * top_k, K/2] 16-byte, [.., K/16] 4-byte aligned, one float
 *   wpacked, wg  packed with gated == 0 ([experts, N, K]), [experts] FP32
 *   weights      device, [tokens, top_k] FP32;  places: the plan's
 *   y            device, [tokens, N] FP32, 16-byte aligned (written)
 *   workspace    device scratch of nvfp4_moe_down_workspace_bytes bytes (0 up to 64 tokens), 256-byte aligned; no state
 */
size_t nvfp4_moe_down_workspace_bytes(int tokens, int top_k, int experts, int N, int K);

nvfp4_status nvfp4_moe_down(const uint8_t* hq, const uint8_t* hs, const float* hg, int tokens, int top_k,
                            const int32_t* offsets, const int32_t* pairs, const int32_t* places, const float* weights,
                            const uint8_t* wpacked, const float* wg, int experts, int N, int K, float* y, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Rules on the logits                                                        */
/* ------------------------------------------------------------------------ */
/*
 * Penalties, biases and grammar masks on logits, in front of the sampler (the
 * ReSET pages run their sampler as a logits processor inside a serving engine,
 * reading note §4.3; these rules are the engine's).  For row r, token v, in
 * this order, each step FP32 with IEEE rounding:
 *   x = logits[r, v]
 *   if v stands in the row's tokens:       x = x > 0 ? x / repetition[r] : x * repetition[r]
 *   c = its count behind the prompt:       x = x - frequency[r] * c;  if c > 0: x = x - presence[r]
 *   if v stands in the row's bias list:    x = x + its value
 *   if the row's grammar forbids v:        x = fill
 * -inf and NaN logits pass through the arithmetic as they are.
 *   logits    device, [rows, V] of dtype NVFP4_DTYPE_*, row r at logits + r * ld (elements)
 *   rows      >= 0;  V 1 .. 2^24;  ld >= V
 *   tokens    device, [rows, history] int32: prompt then output of each row; ids outside [0, V) count nothing.
 *             NULL with history 0: no penalties
 *   n_tokens  device, [rows] int32: how many of them are there (cut to [0, history])
 *   n_prompt  device, [rows] int32: how many of those are the prompt, or NULL: none
 *   repetition, presence, frequency   device, [rows] FP32, each may be NULL (1, 0, 0)
 *   bias_ids, bias_values   device, [rows, n_bias] int32 / FP32 (NULL with n_bias 0); an id outside [0, V) is
 *             an unused entry; of equal ids in a row the last one holds
 *   mask      device, bit v % 32 of word v / 32 set: v is allowed; [mask_count, ceil(V/32)] uint32, or NULL
 *   mask_rows device, [rows] int32: the mask row of each row, -1 (or any outside [0, mask_count)): none;
 *             NULL: row r has mask row r (mask_count >= rows)
 *   fill      what forbidden logits become, e.g. -inf (a row whose mask allows nothing is all fill; reset_sample gives
 *             no token for a row of -inf)
 *   out       device, [rows, V] FP32, 16-byte aligned when V % 4 == 0 is to be fast (written); for FP32 logits with
 *             ld == V it may be the logits themselves
 */
nvfp4_status nvfp4_process_logits(const void* logits, int dtype, int rows, int V, int64_t ld, const int32_t* tokens,
                                  int history, const int32_t* n_tokens, const int32_t* n_prompt,
                                  const float* repetition, const float* presence, const float* frequency,
                                  const int32_t* bias_ids, const float* bias_values, int n_bias, const uint32_t* mask,
                                  int mask_count, const int32_t* mask_rows, float fill, float* out,
                                  cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* ReSET sampler                                                              */
/* ------------------------------------------------------------------------ */
/* Threshold policies (reset_params.threshold).  ReSET's own is the default;
 * the other two are the policies the ReSET reading note compares it with
 * (§3.1 Eq. (1) and §6.3 Table 2).  The sliding-window threshold is read as
 * the mean of the last w token entropies including H, across step boundaries
 * (the pages name the policy without writing it out). */
enum {
  RESET_THRESHOLD_RESET = 0,   /* tau = tau0 if H_step <= H_bar else H_step (SAT over HSE) */
  RESET_THRESHOLD_FIXED = 1,   /* tau = tau0 at every position (Eq. (1))                   */
  RESET_THRESHOLD_WINDOW = 2   /* tau = mean of the last w entropies, including H          */
};

/* A zero-initialised tail (threshold 0, top_p 0) gives ReSET without top-p. */
typedef struct reset_params {
  float tau0;    /* global entropy threshold (nats), used in confident steps        */
  float t_low;   /* temperature below the threshold, > 0                            */
  float t_high;  /* temperature at or above the threshold, > 0                      */
  int w;         /* HSE window: positions 0..w-1 of a step use the last-w mean, 1..256 */
  int threshold; /* RESET_THRESHOLD_*                                                */
  float top_p;   /* nucleus mass in (0, 1); 0 or 1: no truncation                   */
} reset_params;

/* Bytes of the per-row sampler state for M rows and window w. */
size_t reset_state_bytes(int M, int w);

/* Puts every row of `state` at sequence position 0 (asynchronous). */
nvfp4_status reset_state_init(void* state, int M, int w, cudaStream_t stream);

/* The same for the rows r with rows[r] != 0 alone (device, [M] uint8), e.g. where a new request takes a row. */
nvfp4_status reset_state_init_rows(void* state, int M, int w, const uint8_t* rows, cudaStream_t stream);

/* Scratch needed by reset_sample for M rows of V logits. */
size_t reset_workspace_bytes(int M, int V);

/*
 * One decode position of the ReSET sampler for M rows (ReSET reading note
 * §4.1 SAT, §4.2 HSE, §4.3; project page "Step-aware temperature scaling"):
 *   H      = entropy (nats, temperature 1) of softmax(logits[r, :]);
 *   a new step starts at this position when step_start[r] != 0 (the previous
 *   token was the step delimiter) and always at the row's first position;
 *   H_step = mean of the last w entropies (including H) while the in-step
 *            position j < w, else the mean of the step's entropies so far;
 *   H_bar  = mean of all entropies of the row so far (including H);
 *   tau    = tau0 if H_step <= H_bar else H_step   (p->threshold RESET_THRESHOLD_RESET;
 *            tau0 for _FIXED, the mean of the last w entropies for _WINDOW);
 *   T      = t_low if H < tau else t_high;
 *   token  = min{ i : sum_{k<=i} exp((l_k - max l)/T) > u[r] * sum_k exp((l_k - max l)/T) }.
 * With 0 < p->top_p < 1 (reading note §6.1: the evaluation samples with
 * top-p 0.95), the sums run over the nucleus only: token i stays iff the sum
 * of exp((l_k - max l)/T) over the logits l_k > l_i is below top_p times the
 * full sum -- the smallest set of most probable tokens that reaches top_p,
 * with every logit tied to its least probable member.  The top-p path adds
 * four launches and computes in integer masses, exp((l - max l)/T) scaled by
 * 2^(62 - ceil(log2 V)) and rounded: deterministic, accurate to ~1e-7 of Z.
 *
 *   logits     device, [M, V] FP32, 16-byte aligned, finite or -inf (probability 0, e.g. a token that a grammar
 *              forbids).  A row of -inf alone, or with a NaN or +inf, has no distribution: its token is -1, its
 *              H 0 and its T t_high, its state stays as it is, and device error bit 4 is recorded
 *   M          1..64;  V 1 .. 2^24
 *   step_start device, [M] uint8 (may be NULL: no step boundaries)
 *   u          device, [M] FP32 uniforms in [0, 1)
 *   state      device, reset_state_bytes(M, p->w) bytes from reset_state_init (updated)
 *   p          HOST pointer to the parameters (copied at the call); threshold
 *              one of RESET_THRESHOLD_*, top_p in [0, 1] (else NVFP4_ERR_RANGE)
 *   token      device, [M] int32 (written)
 *   H_out      device, [M] FP32 entropies (written; may be NULL)
 *   T_out      device, [M] FP32 chosen temperatures (written; may be NULL)
 *   workspace  device scratch of reset_workspace_bytes(M, V) bytes, 256-byte aligned,
 *              ZEROED ONCE before its first use (every call leaves it ready for
 *              the next); calls that overlap on the GPU must use different workspaces.
 */
nvfp4_status reset_sample(const float* logits, int M, int V, const uint8_t* step_start,
                          const float* u, void* state, const reset_params* p, int32_t* token,
                          float* H_out, float* T_out, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream);

/*
 * reset_sample for the rows r with rows[r] != 0 alone (device, [M] uint8): the
 * others' logits are not read, their state and their entries of token, H_out
 * and T_out stay as they are.  For batches with rows that hold no request.
 */
nvfp4_status reset_sample_rows(const float* logits, int M, int V, const uint8_t* step_start, const float* u,
                               const uint8_t* rows, void* state, const reset_params* p, int32_t* token,
                               float* H_out, float* T_out, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * reset_sample without a workspace argument: same inputs, outputs and rule as
 * reset_sample.  The ReSET pages have no counterpart to this function; it is
 * for callers that cannot allocate device memory -- for example a plugin
 * inside a serving engine that owns every device allocation through its own
 * pool and only hands out fixed input/output buffers, or a latency-critical
 * decode loop that must not call cudaMalloc because it synchronizes the device.
 *
 * Rows of up to 262,144 logits (one thread-block cluster a row, with or
 * without top-p) need no scratch.  Longer rows take a multi-launch path whose
 * scratch (per-row counters, per-chunk partial sums, the top-p records and
 * histograms) lives in a 1,217,280-byte array that the library reserves
 * statically on every GPU that loads it, until the process exits.  Nothing is
 * allocated: no cudaMalloc, cudaFree or allocating library routine.
 *   Limit (V > 262,144 only): M * ceil(V / 2048) <= 4096 (M = 8 allows V up
 *          to 1,048,576); larger calls return NVFP4_ERR_SHAPE without
 *          launching anything.
 *   The first call on a device looks up that device's copy of the array
 *   (cudaGetSymbolAddress); make it before any stream capture on that device.
 *   Every call with V > 262,144 uses the same array and clears its counters
 *   (a 256-byte memset on `stream`); such calls that overlap on the GPU (for
 *   example on two unordered streams) race and give wrong results -- order
 *   them.
 */
nvfp4_status reset_sample_noalloc(const float* logits, int M, int V, const uint8_t* step_start,
                                  const float* u, void* state, const reset_params* p, int32_t* token,
                                  float* H_out, float* T_out, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_GB300_H */
