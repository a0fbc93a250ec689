// pa_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// For each sequence whose context is longer than `budget` rows, every KV head keeps
// `budget` of its rows: those of the `sinks` first and the `recent` last positions,
// and of the others the ones with the highest scores (ties: the lowest row).  A KV
// head's choice is its own: a block-table entry names a block for all KV heads, but
// each head's rows of it are separate memory, so heads may hold different positions
// in the same row.  ("LLM推理与服务：面试问题与推荐回答" Q4: drop the tokens that draw
// little attention.)
//
// Keys.  A row's score as an unsigned integer whose order is the floats' order; NaN
// below every number; a protected position above all.  Kept = the `budget` largest
// (key, then lower row).  The budget-th largest key is found by a radix select, eight
// bits at a time, over keys held in shared memory.
//
// Moves.  Attention does not depend on the order of cached rows (K rows carry their
// rotation), so nothing is shifted: with m rows evicted below `budget`, exactly m kept
// rows lie at or past it, and the i-th of these is copied into the i-th hole.  Sources
// are never written and holes never read, so the copies need no order, and repeating
// the call repeats the same copies.
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKeyCap = 48 * 1024;  // keys held in shared memory (192 KiB)
constexpr uint32_t kProtected = 0xffffffffu;

struct EvictArgs {
  uint8_t *k_cache, *v_cache;
  const float *scores;
  const int32_t *row_pos;
  float *scores_out;
  int32_t *row_pos_out, *new_lens;
  const int32_t *block_tables, *context_lens, *seq_lens;
  int32_t *moves;  // workspace: (hole, source) pairs, list_cap per (sequence, head)
  int num_kv_heads, block_size, max_blocks_per_seq, num_blocks, max_rows;
  int budget, sinks, recent, list_cap, key_cap;
  int row_chunks;  // 16-byte chunks of a cached row
  unsigned *err;
};

__device__ __forceinline__ uint32_t key_of(float score, int pos, int sinks, int64_t recent_from) {
  if (pos < sinks || pos >= recent_from) return kProtected;
  if (score != score) return 0u;
  const uint32_t b = __float_as_uint(score + 0.f);  // (-0 counts as 0)
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive prefix of per-warp values x (all lanes of a warp hold the same x) over the
// CTA's warps; *total = their sum.
__device__ __forceinline__ int warps_before(int x, int *buf, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int y = buf[w];
    before += w < warp ? y : 0;
    all += y;
  }
  *total = all;
  return before;
}

// One CTA per (sequence, KV head).
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int hist[256];
  __shared__ int s_warp[kWarps];
  __shared__ int s_digit, s_left;
  pa::griddep_wait();
  pa::griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seq = blockIdx.x / a.num_kv_heads, head = blockIdx.x % a.num_kv_heads;
  int L = max(0, __ldg(a.context_lens + seq));
  if (L > a.max_rows) {  // context longer than its table
    if (tid == 0 && head == 0) pa::record_error(a.err, pa::kErrCheck);
    L = a.max_rows;
  }
  if (tid == 0 && head == 0) a.new_lens[seq] = min(L, a.budget);
  const int64_t led = ((int64_t)seq * a.num_kv_heads + head) * a.max_rows;
  const float *scores = a.scores + led;
  const int32_t *row_pos = a.row_pos + led;
  float *scores_out = a.scores_out + led;
  int32_t *row_pos_out = a.row_pos_out + led;
  const bool in_place = a.scores == a.scores_out;
  if (L <= a.budget) {
    if (!in_place)
      for (int r = tid; r < L; r += kThreads) {
        scores_out[r] = scores[r];
        row_pos_out[r] = row_pos[r];
      }
    return;
  }
  const int64_t recent_from = (int64_t)__ldg(a.seq_lens + seq) - a.recent;
  auto load_key = [&](int r) { return key_of(scores[r], row_pos[r], a.sinks, recent_from); };
  const int held = min(L, a.key_cap);
  for (int r = tid; r < held; r += kThreads) s_keys[r] = load_key(r);
  auto key = [&](int r) { return r < held ? s_keys[r] : load_key(r); };

  // radix select of the budget-th largest key, from the top byte down: `prefix` holds
  // the bytes known so far, `left` how many rows with that prefix are still to keep
  uint32_t prefix = 0;
  int left = a.budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int r = tid; r < L; r += kThreads) {
      const uint32_t k = key(r);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l takes digits 255 - 8 l .. 248 - 8 l, highest first
      int part = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) part += hist[255 - 8 * lane - i];
      int incl = part;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      int run = incl - part;
      if (run < left && incl >= left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = 255 - 8 * lane - i, n = hist[d];
          if (run < left && run + n >= left) {
            s_digit = d;
            s_left = left - run;
          }
          run += n;
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_digit << shift;
    left = s_left;
    __syncthreads();
  }
  const uint32_t border = prefix;  // rows above it are kept, and the first `left` equal to it

  // each warp takes a contiguous range of rows, in order
  const int per = ((L + kWarps - 1) / kWarps + 31) & ~31;
  const int lo = min(L, warp * per), hi = min(L, lo + per);
  int ties = 0;
  for (int r = lo; r < hi; r += 32)
    ties += __popc(__ballot_sync(0xffffffffu, r + lane < hi && key(r + lane) == border));
  int all;
  const int ties_before = warps_before(ties, s_warp, &all);
  const unsigned below = (1u << lane) - 1u;
  // holes (evicted rows below the budget) and sources (kept rows from there on)
  int32_t *moves = a.moves + ((int64_t)seq * a.num_kv_heads + head) * a.list_cap * 2;
  int holes_at = 0, srcs_at = 0, m = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int t = ties_before, nh = holes_at, ns = srcs_at;
    for (int r0 = lo; r0 < hi; r0 += 32) {
      const int r = r0 + lane;
      const uint32_t k = r < hi ? key(r) : 0u;
      const unsigned eq = __ballot_sync(0xffffffffu, r < hi && k == border);
      const bool kept = r < hi && (k > border || (k == border && t + __popc(eq & below) < left));
      t += __popc(eq);
      const unsigned hb = __ballot_sync(0xffffffffu, r < hi && !kept && r < a.budget);
      const unsigned sb = __ballot_sync(0xffffffffu, kept && r >= a.budget);
      if (pass == 1) {
        if ((hb >> lane) & 1u) moves[2 * (nh + __popc(hb & below))] = r;
        if ((sb >> lane) & 1u) moves[2 * (ns + __popc(sb & below)) + 1] = r;
        if (!in_place && kept && r < a.budget) {
          scores_out[r] = scores[r];
          row_pos_out[r] = row_pos[r];
        }
      }
      nh += __popc(hb);
      ns += __popc(sb);
    }
    if (pass == 0) {
      holes_at = warps_before(nh, s_warp, &all);
      srcs_at = warps_before(ns, s_warp, &m);
    }
  }
  __syncthreads();

  // the copies: a warp per pair, lanes over its chunks (K, then V)
  const int rc = a.row_chunks;
  const int32_t *table = a.block_tables + (int64_t)seq * a.max_blocks_per_seq;
  for (int i = warp; i < m; i += kWarps) {
    const int to = moves[2 * i], from = moves[2 * i + 1];
    if (lane == 0) {
      scores_out[to] = scores[from];
      row_pos_out[to] = row_pos[from];
    }
    const int bt = __ldg(table + to / a.block_size), bf = __ldg(table + from / a.block_size);
    if (bt < 0 || bt >= a.num_blocks || bf < 0 || bf >= a.num_blocks) {
      if (lane == 0) pa::record_error(a.err, pa::kErrCheck);
      continue;
    }
    const int64_t rt = ((int64_t)bt * a.num_kv_heads + head) * a.block_size + to % a.block_size;
    const int64_t rf = ((int64_t)bf * a.num_kv_heads + head) * a.block_size + from % a.block_size;
    for (int c = lane; c < 2 * rc; c += 32) {
      uint8_t *cache = c < rc ? a.k_cache : a.v_cache;
      const int cc = c < rc ? c : c - rc;
      const uint4 x = *(reinterpret_cast<const uint4 *>(cache) + rf * rc + cc);
      *(reinterpret_cast<uint4 *>(cache) + rt * rc + cc) = x;
    }
  }
}

}  // namespace

extern "C" PA_API size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int budget) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || budget <= 0) return 0;
  return (size_t)num_seqs * num_kv_heads * budget * 2 * sizeof(int32_t);
}

extern "C" PA_API pa_status pa_evict(
    void *k_cache, void *v_cache, float *scores_out, int32_t *row_pos_out, int32_t *new_lens,
    const float *scores, const int32_t *row_pos, const int32_t *block_tables,
    const int32_t *context_lens, const int32_t *seq_lens, int num_seqs, int num_kv_heads,
    int head_dim, int block_size, int max_blocks_per_seq, int num_blocks, int budget, int sinks,
    int recent, int element_bytes, void *workspace, size_t workspace_bytes, void *stream) {
  if (!k_cache || !v_cache || !scores_out || !row_pos_out || !new_lens || !scores || !row_pos ||
      !block_tables || !context_lens || !seq_lens || !workspace)
    return PA_ERR_INVALID_ARG;
  if (num_seqs <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (budget <= 0 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return PA_ERR_INVALID_ARG;
  // the ledgers are both updated in place or both written elsewhere
  if ((scores == scores_out) != (row_pos == row_pos_out)) return PA_ERR_INVALID_ARG;
  if (new_lens == context_lens) return PA_ERR_INVALID_ARG;  // (every KV head reads the old lengths)
  if (!pa::aligned16(k_cache) || !pa::aligned16(v_cache) || !pa::aligned16(workspace))
    return PA_ERR_INVALID_ARG;
  if (element_bytes != 1 && element_bytes != 2) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (element_bytes == 1 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (!pa::supported_block(block_size)) return PA_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size >= (int64_t)1 << 30) return PA_ERR_INVALID_ARG;
  if ((int64_t)num_seqs * num_kv_heads >= (int64_t)1 << 31) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < pa_evict_workspace_size(num_seqs, num_kv_heads, budget))
    return PA_ERR_INVALID_ARG;
  EvictArgs a;
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.scores = scores;
  a.row_pos = row_pos;
  a.scores_out = scores_out;
  a.row_pos_out = row_pos_out;
  a.new_lens = new_lens;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.seq_lens = seq_lens;
  a.moves = static_cast<int32_t *>(workspace);
  a.num_kv_heads = num_kv_heads;
  a.block_size = block_size;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.max_rows = max_blocks_per_seq * block_size;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.list_cap = budget;
  a.key_cap = std::min(a.max_rows, kKeyCap);
  a.row_chunks = head_dim * element_bytes / 16;
  a.err = pa::error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  const int smem = a.key_cap * (int)sizeof(uint32_t);
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kKeyCap * (int)sizeof(uint32_t)) != cudaSuccess)
    return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_seqs * num_kv_heads), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
