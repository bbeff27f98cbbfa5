// Page tables and slot maps of a paged KV cache, built on the GPU from the
// requests' lengths, and the return of ended requests' pages.
//
// Both operators are a prefix sum over the requests (pages needed or given
// back; new tokens) followed by a flat loop over what it counts (pages, tokens),
// each item finding its request by a binary search in the sums.  They are bound
// by latency: a few dependent L2 round trips (lengths -> sums -> table or stack
// -> slot) in one launch.  Every CTA therefore forms the sums of all requests
// by itself -- at 1024 requests two coalesced loads and one block scan --
// instead of waiting for another CTA's, and takes its share of the flat loops.
// 8 decoding requests: 4.3 us for release and plan in a graph; 1024 requests, half of
// them prompts, 187000 tokens: 14.3 us.  The plan alone of the latter, call after call, takes
// 7.6 us, 4.0 with no new token (a launch and the sums: 2.6 for 8 requests, 5.0 for 1024 with
// a token each), the release alone 3.7.
#include "common.cuh"

namespace {

constexpr int kMaxThreads = 1024;
// Tokens or pages a CTA has before another is worth its own scan: 64 requests of 64 to 256 new tokens each took 5.6 us
// with 256, 7.2 with 1024, 10.2 with 2048, 30 with 8192; new tokens of decoding requests fit one CTA's share anyway.
constexpr int kItems = 256;

// Inclusive block scan of two counters at once; tot = the block's totals.
template <int THREADS>
NVFP4_DEVINL int2 block_scan(int2 v, int2* s_warp, int2& tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, v.x, o), b = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += a;
      v.y += b;
    }
  }
  __syncthreads();                       // the previous tile's sums have been read
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int2 w = lane < THREADS / 32 ? s_warp[lane] : make_int2(0, 0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, w.x, o), b = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += a;
      w.y += b;
    }
  }
  tot = make_int2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
  if (warp > 0) {
    v.x += __shfl_sync(0xffffffffu, w.x, warp - 1);
    v.y += __shfl_sync(0xffffffffu, w.y, warp - 1);
  }
  return v;
}

// Largest i in [0, n) with s[i] <= x (s non-decreasing, s[0] <= x).
NVFP4_DEVINL int find_le(const int* s, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

struct PlanArgs {
  const int32_t *ctx, *add;
  int32_t* table;
  const int32_t *stack, *count;
  int32_t *count_out, *kv_lens, *cu_q, *slots, *positions, *info;
  int batch, page, width, capacity, max_tokens;
  int count_only;                        // write count_out and kv_lens (where they are not NULL) and nothing else
};

template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv_plan_kernel(const PlanArgs a) {
  __shared__ int2 s_warp[32];
  __shared__ int s_tok[THREADS];         // a tile's first token of each request
  __shared__ int s_pg[THREADS];          // pages needed before each request
  __shared__ int s_ctx[THREADS];         // ~ctx for a refused request
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const int avail = min(max(*a.count, 0), a.capacity);
  const int t_lo = (int)((long long)a.max_tokens * blockIdx.x / gridDim.x);
  const int t_hi = (int)((long long)a.max_tokens * (blockIdx.x + 1) / gridDim.x);
  int tok0 = 0, pg0 = 0, taken = 0, refused = 0;
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    const int b = b0 + tid;
    int c = 0, q = 0, need = 0, bad = 0;
    if (b < a.batch) {
      c = a.ctx[b];
      q = a.add[b];
      bad = c < 0 || q < 0;
      c = max(c, 0);
      q = max(q, 0);
      const long long end = ((long long)c + q + a.page - 1) / a.page;
      bad = bad || end > a.width;
      need = bad ? 0 : (int)end - (int)(((long long)c + a.page - 1) / a.page);
    }
    int2 tot;
    const int2 inc = block_scan<THREADS>(make_int2(q, need), s_warp, tot);
    const int refuse = bad || (need > 0 && pg0 + inc.y > avail);
    s_tok[tid] = tok0 + inc.x - q;
    s_pg[tid] = pg0 + inc.y - need;
    s_ctx[tid] = refuse ? ~c : c;
    refused += __syncthreads_count(refuse && b < a.batch);
    const int tok_end = tok0 + tot.x;
    const int n = min(THREADS, a.batch - b0);
    if (a.kv_lens && blockIdx.x == 0 && b < a.batch) a.kv_lens[b] = refuse ? c : c + q;
    if (!a.count_only) {
      if (blockIdx.x == 0 && b < a.batch) {
        a.cu_q[b] = s_tok[tid];
        if (b == a.batch - 1) a.cu_q[a.batch] = tok_end;
      }
      // this CTA's share of the tile's new pages
      const int p_end = min(pg0 + tot.y, avail);
      for (int i = pg0 + blockIdx.x * THREADS + tid; i < p_end; i += gridDim.x * THREADS) {
        const int r = find_le(s_pg, n, i);
        const int ctx = s_ctx[r];
        if (ctx >= 0)
          a.table[(size_t)(b0 + r) * a.width + (ctx + a.page - 1) / a.page + (i - s_pg[r])] = a.stack[avail - 1 - i];
      }
      // and of its new tokens
      for (int t = max(t_lo, tok0) + tid; t < min(t_hi, tok_end); t += THREADS) {
        const int r = find_le(s_tok, n, t);
        const int v = s_ctx[r], ctx = v < 0 ? ~v : v;
        const int pos = ctx + (t - s_tok[r]);
        int slot = -1;
        if (v >= 0) {
          const int held = (ctx + a.page - 1) / a.page, j = pos / a.page;
          const int from = avail - 1 - (s_pg[r] + j - held);
          // both in range unless the token counts of a call sum past 2^31
          if (j >= 0 && j < a.width && (j < held || (from >= 0 && from < avail))) {
            const int page = j < held ? a.table[(size_t)(b0 + r) * a.width + j] : a.stack[from];
            slot = page * a.page + (pos - j * a.page);
          }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
      }
    }
    // pages taken so far: the inclusive sum of the last served request that needs any (needs are summed in
    // request order, so the served ones come before the refused ones)
    const int mine = !refuse && need > 0 ? pg0 + inc.y : 0;
    int m = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();
    if ((tid & 31) == 0) s_warp[tid >> 5].x = m;
    __syncthreads();
    for (int w = 0; w < THREADS / 32; ++w) taken = max(taken, s_warp[w].x);
    tok0 = tok_end;
    pg0 += tot.y;
  }
  if (!a.count_only) {
    for (int t = max(t_lo, tok0) + tid; t < t_hi; t += THREADS) {
      a.slots[t] = -1;
      a.positions[t] = 0;
    }
    if (blockIdx.x == 0 && tid == 0) {
      a.info[0] = refused;
      a.info[1] = tok0;
    }
  }
  if (a.count_out && blockIdx.x == 0 && tid == 0) *a.count_out = avail - taken;
}

struct ReleaseArgs {
  const int32_t* lens;
  const uint8_t* ended;
  const int32_t* table;
  int32_t* stack;
  const int32_t* count;
  int32_t* count_out;
  int batch, page, width, capacity;
  int count_only;
};

__global__ void __launch_bounds__(kMaxThreads) kv_release_kernel(const ReleaseArgs a) {
  __shared__ int2 s_warp[32];
  __shared__ int s_pg[kMaxThreads];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const int have = min(max(*a.count, 0), a.capacity);
  int pg0 = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kMaxThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < a.batch && a.ended[b] != 0) {
      const int len = max(a.lens[b], 0);
      n = (int)min(((long long)len + a.page - 1) / a.page, (long long)a.width);
    }
    int2 tot;
    const int2 inc = block_scan<kMaxThreads>(make_int2(n, 0), s_warp, tot);
    s_pg[tid] = pg0 + inc.x - n;
    __syncthreads();
    if (!a.count_only) {
      const int end = min(pg0 + tot.x, a.capacity - have);
      for (int i = pg0 + blockIdx.x * kMaxThreads + tid; i < end; i += gridDim.x * kMaxThreads) {
        const int r = find_le(s_pg, min(kMaxThreads, a.batch - b0), i);
        a.stack[have + i] = a.table[(size_t)(b0 + r) * a.width + (i - s_pg[r])];
      }
    }
    pg0 += tot.x;
  }
  if (a.count_out && blockIdx.x == 0 && tid == 0) *a.count_out = have + min(pg0, a.capacity - have);
}

template <class Args>
cudaError_t launch(void (*kern)(Args), int grid, int threads, const Args& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// CTAs that may start after others have ended must not read a count that those
// have written: with several CTAs and one address for both counts, the count
// is written by a second launch of one CTA.  So are the new lengths of a plan
// that lie over the old ones.
cudaError_t launch_counted(void (*kern)(ReleaseArgs), int grid, int threads, ReleaseArgs a, cudaStream_t stream) {
  const bool split = grid > 1 && a.count_out == a.count;
  int32_t* out = a.count_out;
  if (split) a.count_out = nullptr;
  cudaError_t e = launch(kern, grid, threads, a, stream);
  if (e == cudaSuccess && split) {
    a.count_out = out;
    a.count_only = 1;
    e = launch(kern, 1, threads, a, stream);
  }
  return e;
}
cudaError_t launch_counted(void (*kern)(PlanArgs), int grid, int threads, PlanArgs a, cudaStream_t stream) {
  PlanArgs later = a;
  later.count_only = 1;
  if (grid == 1 || a.count_out != a.count) later.count_out = nullptr;
  else a.count_out = nullptr;
  if (grid == 1 || a.kv_lens != a.ctx) later.kv_lens = nullptr;
  else a.kv_lens = nullptr;
  cudaError_t e = launch(kern, grid, threads, a, stream);
  if (e == cudaSuccess && (later.count_out || later.kv_lens)) e = launch(kern, 1, threads, later, stream);
  return e;
}

struct Range {
  const void* p;
  size_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.bytes && y < x + a.bytes;
}

bool page_ok(int page_size) { return page_size >= 16 && page_size <= 1024 && page_size % 16 == 0; }

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

extern "C" nvfp4_status nvfp4_kv_release(const int32_t* lens, const uint8_t* ended, int batch, int page_size,
                                         const int32_t* block_table, int table_width, int32_t* free_pages,
                                         int free_capacity, const int32_t* free_count, int32_t* free_count_out,
                                         cudaStream_t stream) {
  if ((!free_pages && free_capacity > 0) || !free_count || !free_count_out) return NVFP4_ERR_NULL;
  if (batch > 0 && (!lens || !ended || !block_table)) return NVFP4_ERR_NULL;
  if (batch < 0 || table_width < 0 || free_capacity < 0) return NVFP4_ERR_SHAPE;
  if (!page_ok(page_size)) return NVFP4_ERR_SHAPE;
  if ((long long)batch * table_width > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  for (const void* p : {(const void*)lens, (const void*)block_table, (const void*)free_pages, (const void*)free_count,
                        (const void*)free_count_out})
    if (!nvfp4_internal_aligned(p, 4)) return NVFP4_ERR_ALIGN;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  const ReleaseArgs a = {lens, ended, block_table, free_pages, free_count, free_count_out,
                         batch, page_size, table_width, free_capacity, 0};
  const long long most = (long long)batch * table_width;
  const int grid = (int)(most < kItems ? 1 : most / kItems < 64 ? most / kItems : 64);
  return nvfp4_internal_cuda_status(launch_counted(kv_release_kernel, grid, kMaxThreads, a, stream));
}

extern "C" nvfp4_status nvfp4_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int batch, int page_size,
                                      int32_t* block_table, int table_width, const int32_t* free_pages,
                                      int free_capacity, const int32_t* free_count, int32_t* free_count_out,
                                      int32_t* kv_lens, int32_t* cu_q, int32_t* slots, int32_t* positions,
                                      int max_tokens, int32_t* info, cudaStream_t stream) {
  if (!ctx_lens || !new_lens || !block_table || (!free_pages && free_capacity > 0) || !free_count ||
      !free_count_out || !kv_lens || !cu_q || !info)
    return NVFP4_ERR_NULL;
  if (max_tokens > 0 && (!slots || !positions)) return NVFP4_ERR_NULL;
  if (batch < 1 || table_width < 1 || free_capacity < 0 || max_tokens < 0) return NVFP4_ERR_SHAPE;
  if (!page_ok(page_size) || (long long)batch * table_width > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  for (const void* p : {(const void*)ctx_lens, (const void*)new_lens, (const void*)block_table,
                        (const void*)free_pages, (const void*)free_count, (const void*)free_count_out,
                        (const void*)kv_lens, (const void*)cu_q, (const void*)slots, (const void*)positions,
                        (const void*)info})
    if (!nvfp4_internal_aligned(p, 4)) return NVFP4_ERR_ALIGN;
  {
    // what is written, then what is read only; kv_lens over ctx_lens and free_count_out over free_count are allowed
    const size_t n = (size_t)batch * 4, t = (size_t)max_tokens * 4;
    const Range r[] = {{kv_lens, n}, {free_count_out, 4}, {block_table, n * table_width}, {cu_q, n + 4}, {slots, t},
                       {positions, t}, {info, 8}, {ctx_lens, n}, {free_count, 4}, {new_lens, n},
                       {free_pages, (size_t)free_capacity * 4}};
    for (int i = 0; i < 7; ++i)
      for (int j = i + 1; j < 11; ++j)
        if (r[i].bytes && r[j].bytes && overlap(r[i], r[j]) && !(j == i + 7 && i < 2 && r[i].p == r[j].p))
          return NVFP4_ERR_SHAPE;
  }
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  const PlanArgs a = {ctx_lens, new_lens, block_table, free_pages, free_count, free_count_out, kv_lens, cu_q, slots,
                      positions, info, batch, page_size, table_width, free_capacity, max_tokens, 0};
  const int grid = max_tokens < kItems ? 1 : max_tokens / kItems < 152 ? max_tokens / kItems : 152;
  // (batch 32 with 256 / 1024 threads: 4.4 / 5.5 us, 256: 5.2 / 6.3;  512: 7.5 / 6.5, 1024: 12.1 / 7.2)
  const cudaError_t e = batch <= 256 ? launch_counted(kv_plan_kernel<256>, grid, 256, a, stream)
                                     : launch_counted(kv_plan_kernel<kMaxThreads>, grid, kMaxThreads, a, stream);
  return nvfp4_internal_cuda_status(e);
}
