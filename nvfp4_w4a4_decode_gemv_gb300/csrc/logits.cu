// Rules on the logits in front of the sampler: penalties for tokens that
// occurred, biases and grammar masks, in one pass.
//
// A row's counts, its bias entries and its mask all belong to token ids, so the
// vocabulary is cut into chunks, one CTA each.  A CTA asks for its logits first
// (16 or 4 a thread, in registers), counts the row's tokens that fall into its
// chunk in shared memory while they come (integer atomics: any order gives the
// same counts), applies the penalties, marks the last bias entry of each id in the
// same memory (an integer maximum), and writes each logit once.  Bound by HBM for
// large batches (4 bytes in, 4 out a logit), by latency for small ones.  Every
// CTA of a row reads the row's whole history (from L2): 16 KB against the 64 KB of
// logits of an 8192-token chunk at 4096 tokens.  64 rows of 151936 logits: 19 us with
// 256 tokens a row (12.2 at the copy rate), 31 with 16384: the rest is issue slots of the
// looks at tokens, and the shared atomics of the first chunks, which hold most of them.  Counted once a cluster of 7 CTAs, through their distributed
// shared memory, it took 50 us (30 instead of 20 with 256 tokens a row).
#include <math.h>

#include "common.cuh"

namespace {

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
  int V, history, n_bias, mask_count;
  int vec_in, vec_out, vec_tok;             // rows can be read / written / scanned in whole 4-element pieces
};

NVFP4_DEVINL float load1(const float* p) { return *p; }
NVFP4_DEVINL float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
NVFP4_DEVINL float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
NVFP4_DEVINL float4 load4(const uint16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

// PIECES pieces of 4 logits a thread: a chunk of 4 * PIECES * THREADS.
template <class T, int THREADS, int PIECES>
__global__ void __launch_bounds__(THREADS) process_logits_kernel(const LogitArgs a) {
  constexpr int kChunk = 4 * PIECES * THREADS;
  __shared__ __align__(16) uint32_t s_tab[kChunk];
  griddep_launch_dependents();
  const int r = blockIdx.x, tid = threadIdx.x;
  const int v0 = blockIdx.y * kChunk;
  const int n = min(kChunk, a.V - v0);
#pragma unroll
  for (int k = 0; k < PIECES; ++k) *reinterpret_cast<uint4*>(&s_tab[4 * (tid + k * THREADS)]) = make_uint4(0u, 0u, 0u, 0u);
  griddep_wait();
  const T* in = static_cast<const T*>(a.logits) + (size_t)r * a.ld + v0;
  float x[PIECES][4];
#pragma unroll
  for (int k = 0; k < PIECES; ++k) {
    const int i = 4 * (tid + k * THREADS);
    if (a.vec_in && i + 4 <= n) {
      const float4 f = load4(in + i);
      x[k][0] = f.x, x[k][1] = f.y, x[k][2] = f.z, x[k][3] = f.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[k][j] = i + j < n ? load1(in + i + j) : 0.0f;
    }
  }
  // everything that waits for no other load is asked for before anything is used: the row's parameters, the first
  // pieces of its history (all of the row's `history` entries exist, however many are in use), its first bias entry
  const int32_t* tok = a.tokens + (size_t)r * a.history;
  constexpr int kBatch = 4;                 // pieces of history in flight
  int4 q[kBatch];
  if (a.vec_tok) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (tid + j * THREADS < a.history / 4) q[j] = __ldcg(reinterpret_cast<const int4*>(tok) + tid + j * THREADS);
  }
  int used = 0, prompt = 0;
  float rep = 1.0f, pres = 0.0f, freq = 0.0f;
  if (a.history > 0) {
    used = a.n_tokens[r];
    if (a.n_prompt) prompt = a.n_prompt[r];
    if (a.repetition) rep = a.repetition[r];
    if (a.presence) pres = a.presence[r];
    if (a.frequency) freq = a.frequency[r];
  }
  const int32_t* ids = a.bias_ids + (size_t)r * a.n_bias;
  const float* values = a.bias_values + (size_t)r * a.n_bias;
  const int32_t id0 = tid < a.n_bias ? ids[tid] : -1;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_rows ? a.mask_rows[r] : r;
    if (m >= 0 && m < a.mask_count) mask = a.mask + (size_t)m * ((a.V + 31) / 32);
  }
  uint32_t allowed[PIECES];                 // a piece lies in one word: v0 and i are multiples of 4
#pragma unroll
  for (int k = 0; k < PIECES; ++k) {
    const int i = 4 * (tid + k * THREADS);
    allowed[k] = mask && i < n ? mask[(v0 + i) >> 5] : ~0u;
  }
  used = min(max(used, 0), a.history);
  prompt = min(max(prompt, 0), used);
  __syncthreads();
  if (a.history > 0) {
    auto count = [&](int32_t id, int i) {
      const uint32_t v = (uint32_t)id - (uint32_t)v0;
      if (v < (uint32_t)n) {
        if (i < prompt) atomicOr(&s_tab[v], kPrompt);
        else atomicAdd(&s_tab[v], 1u);
      }
    };
    int i = 0;
    if (a.vec_tok) {
      const int pieces = used / 4;
      for (int p = tid; p < pieces; p += kBatch * THREADS) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int at = 4 * (p + j * THREADS);
          if (at < 4 * pieces) {
            count(q[j].x, at);
            count(q[j].y, at + 1);
            count(q[j].z, at + 2);
            count(q[j].w, at + 3);
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (p + (kBatch + j) * THREADS < pieces)
            q[j] = __ldcg(reinterpret_cast<const int4*>(tok) + p + (kBatch + j) * THREADS);
      }
      i = 4 * pieces;
    }
    for (i += tid; i < used; i += THREADS) count(__ldcg(tok + i), i);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      const uint4 c4 = *reinterpret_cast<const uint4*>(&s_tab[4 * (tid + k * THREADS)]);
      if (!(c4.x | c4.y | c4.z | c4.w)) continue;
      const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c[j]) {
          const uint32_t times = c[j] & ~kPrompt;
          x[k][j] = x[k][j] > 0.0f ? __fdiv_rn(x[k][j], rep) : __fmul_rn(x[k][j], rep);
          if (times) x[k][j] = __fsub_rn(__fsub_rn(x[k][j], __fmul_rn(freq, (float)times)), pres);
        }
    }
  }
  if (a.n_bias > 0) {
    // the same memory: 1 + the last bias entry of each id, 0 none (a thread clears what it alone has read)
    if (a.history > 0) {
#pragma unroll
      for (int k = 0; k < PIECES; ++k)
        *reinterpret_cast<uint4*>(&s_tab[4 * (tid + k * THREADS)]) = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
    }
    for (int i = tid; i < a.n_bias; i += THREADS) {
      const uint32_t v = (uint32_t)(i == tid ? id0 : ids[i]) - (uint32_t)v0;
      if (v < (uint32_t)n) atomicMax(&s_tab[v], (uint32_t)i + 1u);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      const uint4 c4 = *reinterpret_cast<const uint4*>(&s_tab[4 * (tid + k * THREADS)]);
      const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c[j]) x[k][j] = __fadd_rn(x[k][j], values[c[j] - 1u]);
    }
  }
  float* out = a.out + (size_t)r * a.V + v0;
#pragma unroll
  for (int k = 0; k < PIECES; ++k) {
    const int i = 4 * (tid + k * THREADS);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!((allowed[k] >> ((v0 + i + j) & 31)) & 1u)) x[k][j] = a.fill;
    if (a.vec_out && i + 4 <= n) {
      *reinterpret_cast<float4*>(out + i) = make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) out[i + j] = x[k][j];
    }
  }
}

template <class T, int THREADS, int PIECES>
cudaError_t launch(const LogitArgs& a, int rows, cudaStream_t stream) {
  constexpr int kChunk = 4 * PIECES * THREADS;
  cudaLaunchConfig_t cfg = {};
  // the first chunks of all rows first: vocabularies have their frequent tokens there, so most of the counting (chunk
  // after chunk of one row instead: 32.2 us, not 30.7, for 64 rows with 16384 tokens each)
  cfg.gridDim = dim3((unsigned)rows, (unsigned)((a.V + kChunk - 1) / kChunk));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, process_logits_kernel<T, THREADS, PIECES>, a);
}

template <class T>
cudaError_t dispatch(const LogitArgs& a, int rows, cudaStream_t stream) {
  // large chunks once they fill the GPU, for the history is read over less then: V = 151936, history 2000, small / large
  // chunks: 4 rows (76 CTAs) 4.6 / 5.4 us, 6 rows 4.6 / 5.9, 8 rows 6.4 / 5.4, 16 rows 9.9 / 6.4, 64 rows 33 / 20
  if ((long long)rows * ((a.V + 8191) / 8192) >= 152) return launch<T, 512, 4>(a, rows, stream);
  return launch<T, 256, 1>(a, rows, stream);
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
                 mask, mask_rows, fill, V, history, n_bias, mask_count, 0, 0, 0};
  const size_t piece_in = dtype == NVFP4_DTYPE_F32 ? 16 : 8;       // bytes of 4 logits
  a.vec_in = nvfp4_internal_aligned(logits, piece_in) && (rows == 1 || ld % 4 == 0);
  a.vec_out = nvfp4_internal_aligned(out, 16) && (rows == 1 || V % 4 == 0);
  a.vec_tok = history > 0 && nvfp4_internal_aligned(tokens, 16) && (rows == 1 || history % 4 == 0);
  return nvfp4_internal_cuda_status(dtype == NVFP4_DTYPE_F32 ? dispatch<float>(a, rows, stream)
                                                             : dispatch<uint16_t>(a, rows, stream));
}
