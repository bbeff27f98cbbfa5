// Rules on the logits in front of the sampler: penalties for tokens that
// occurred, biases and grammar masks, in one pass.
//
// A row's counts, its bias entries and its mask all belong to token ids, so the
// vocabulary is cut into chunks: a CTA counts the row's tokens that fall into its
// chunk in shared memory (integer atomics: any order gives the same counts),
// marks the last bias entry of each id (an integer maximum), and then streams its
// logits through once.  Bound by HBM for large batches (4 bytes in, 4 out a
// logit), by latency for small ones.
#include <math.h>

#include "common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kPrompt = 0x80000000u;   // the token stands in the prompt; the other bits count the output

struct LogitArgs {
  const void* logits;
  int64_t ld;
  float* out;
  const int32_t *tokens, *n_tokens, *n_prompt;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_ids;
  const float* bias_values;
  const uint32_t* mask;
  const int32_t* mask_rows;
  float fill;
  int V, history, n_bias, mask_count, chunk;
};

NVFP4_DEVINL float load1(const float* p) { return *p; }
NVFP4_DEVINL float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

template <class T>
__global__ void __launch_bounds__(kThreads) process_logits_kernel(const LogitArgs a) {
  extern __shared__ uint32_t smem[];
  uint32_t* count = smem;                   // [chunk]
  uint32_t* bias = smem + a.chunk;          // [chunk], only with biases: 1 + the last entry of the id, 0 none
  griddep_launch_dependents();
  griddep_wait();
  const int r = blockIdx.y, tid = threadIdx.x;
  const int v0 = blockIdx.x * a.chunk;
  const int n = min(a.chunk, a.V - v0);
  const bool has_tokens = a.history > 0, has_bias = a.n_bias > 0;
  for (int i = tid; i < (has_bias ? 2 : 1) * a.chunk; i += kThreads) smem[i] = 0u;
  __syncthreads();
  if (has_tokens) {
    const int used = min(max(a.n_tokens[r], 0), a.history);
    const int prompt = a.n_prompt ? min(max(a.n_prompt[r], 0), used) : 0;
    const int32_t* tok = a.tokens + (size_t)r * a.history;
    for (int i = tid; i < used; i += kThreads) {
      const uint32_t v = (uint32_t)tok[i] - (uint32_t)v0;
      if (v < (uint32_t)n) {
        if (i < prompt) atomicOr(&count[v], kPrompt);
        else atomicAdd(&count[v], 1u);
      }
    }
  }
  if (has_bias) {
    const int32_t* ids = a.bias_ids + (size_t)r * a.n_bias;
    for (int i = tid; i < a.n_bias; i += kThreads) {
      const uint32_t v = (uint32_t)ids[i] - (uint32_t)v0;
      if (v < (uint32_t)n) atomicMax(&bias[v], (uint32_t)i + 1u);
    }
  }
  __syncthreads();
  const float rep = a.repetition ? a.repetition[r] : 1.0f;
  const float pres = a.presence ? a.presence[r] : 0.0f;
  const float freq = a.frequency ? a.frequency[r] : 0.0f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_rows ? a.mask_rows[r] : r;
    if (m >= 0 && m < a.mask_count) mask = a.mask + (size_t)m * ((a.V + 31) / 32);
  }
  const T* in = static_cast<const T*>(a.logits) + (size_t)r * a.ld + v0;
  float* out = a.out + (size_t)r * a.V + v0;
  for (int i = tid; i < n; i += kThreads) {
    float x = load1(in + i);
    const uint32_t c = count[i];
    if (c) {
      x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
      const uint32_t k = c & ~kPrompt;
      if (k) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, (float)k)), pres);
    }
    if (has_bias && bias[i]) x = __fadd_rn(x, a.bias_values[(size_t)r * a.n_bias + bias[i] - 1u]);
    if (mask && !((mask[(v0 + i) >> 5] >> ((v0 + i) & 31)) & 1u)) x = a.fill;
    out[i] = x;
  }
}

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

extern "C" nvfp4_status nvfp4_process_logits(const void* logits, int dtype, int rows, int V, int64_t ld,
                                             const int32_t* tokens, int history, const int32_t* n_tokens,
                                             const int32_t* n_prompt, const float* repetition, const float* presence,
                                             const float* frequency, const int32_t* bias_ids,
                                             const float* bias_values, int n_bias, const uint32_t* mask,
                                             int mask_count, const int32_t* mask_rows, float fill, float* out,
                                             cudaStream_t stream) {
  if (dtype != NVFP4_DTYPE_F32 && dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_RANGE;
  if (rows < 0 || rows > 65535 || V < 1 || V > (1 << 24) || ld < V || history < 0 || n_bias < 0) return NVFP4_ERR_SHAPE;
  if (mask && (mask_count < 1 || (!mask_rows && mask_count < rows))) return NVFP4_ERR_SHAPE;
  if (rows == 0) return NVFP4_OK;
  if (!logits || !out || (history > 0 && (!tokens || !n_tokens)) || (n_bias > 0 && (!bias_ids || !bias_values)))
    return NVFP4_ERR_NULL;
  for (const void* p : {(const void*)tokens, (const void*)n_tokens, (const void*)n_prompt, (const void*)repetition,
                        (const void*)presence, (const void*)frequency, (const void*)bias_ids,
                        (const void*)bias_values, (const void*)mask, (const void*)mask_rows, (const void*)out})
    if (!nvfp4_internal_aligned(p, 4)) return NVFP4_ERR_ALIGN;
  if (!nvfp4_internal_aligned(logits, dtype == NVFP4_DTYPE_F32 ? 4 : 2)) return NVFP4_ERR_ALIGN;
  if (logits == out && (dtype != NVFP4_DTYPE_F32 || ld != V)) return NVFP4_ERR_SHAPE;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  LogitArgs a = {logits, ld, out, tokens, n_tokens, n_prompt, repetition, presence, frequency, bias_ids, bias_values,
                 mask, mask_rows, fill, V, history, n_bias, mask_count, 0};
  a.chunk = 4096;
  const dim3 grid((unsigned)((V + a.chunk - 1) / a.chunk), (unsigned)rows);
  const size_t smem = (size_t)a.chunk * 4 * (n_bias > 0 ? 2 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return nvfp4_internal_cuda_status(dtype == NVFP4_DTYPE_F32
                                        ? cudaLaunchKernelEx(&cfg, process_logits_kernel<float>, a)
                                        : cudaLaunchKernelEx(&cfg, process_logits_kernel<uint16_t>, a));
}
