// pa_scored.cu -- the ledger of accumulated attention weight: what each cached row
// drew from this step's queries, added to the row's score.
//
// For KV head h of sequence i and cached row t
//   share(t) = sum over the head's query rows r that see t of
//              2^(s_rt - m_r) / l_r                 (s in base-2 units)
// with m_r and l_r the row's softmax maximum and sum.  These are known only after the
// attention pass, so the weights take a second look at the scores:
//   * up to 16 query tokens: the decode pass leaves its scores in the workspace, 4 bytes
//     per query row and cached row against the 2 head_dim 16-bit values per cached row of
//     K and V.  They are read back from L2, by the same CTAs where those hold all of a
//     KV head's rows (pa_decode.cuh), else by ledger_kernel;
//   * more: the scores would outgrow the cache, so mass_tc_kernel (pa_mass_tc.cuh)
//     computes them again from K and q.
// Rows that this step appended (the last q_len) start their scores here, and their
// positions are noted; a row's score is written by one thread, so the sums have one
// order.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "pa_launch.h"
#include "pa_mass_tc.cuh"
#include "pa_scored.h"

namespace pa {

namespace {

constexpr int kLedgerThreads = 256;
constexpr int kRowBatch = 256;  // rows whose statistics are in shared memory at once

// A CTA takes 256 cached rows of one (sequence, KV head).
__global__ void __launch_bounds__(kLedgerThreads) ledger_kernel(const LedgerArgs a) {
  __shared__ float s_m[kRowBatch], s_inv[kRowBatch];
  griddep_wait();
  griddep_launch_dependents();
  const int chunks = (a.max_rows + kLedgerThreads - 1) / kLedgerThreads;
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int seq = unit / a.num_kv_heads, kvh = unit % a.num_kv_heads;
  const int Lc = max(0, __ldg(a.context_lens + seq)), L = min(Lc, a.max_rows);
  if (chunk * kLedgerThreads >= L) return;
  const int t = chunk * kLedgerThreads + threadIdx.x;
  const float *raw = a.raw_scores + ((size_t)unit * a.max_tiles + t / kTileTokens) * a.rows * kTileTokens +
                     t % kTileTokens;
  const int heads = a.group * a.num_kv_heads;
  float share = 0.f;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t at = (int64_t)unit * a.max_rows + t;
  const float old = t < L ? a.scores[at] : 0.f;
  for (int r0 = 0; r0 < a.rows; r0 += kRowBatch) {
    const int n = min(kRowBatch, a.rows - r0);
    __syncthreads();
    for (int r = warp; r < n; r += kLedgerThreads / 32) {
      // a warp merges the partitions' statistics of query token u, head h
      const int u = (r0 + r) / a.group, h = kvh * a.group + (r0 + r) % a.group;
      const size_t base = (size_t)seq * a.splits * a.q_len * heads + (size_t)u * heads + h;
      const size_t step = (size_t)a.q_len * heads;
      float m = -INFINITY;
      for (int p = lane; p < a.splits; p += 32)
        if (a.ws_l[base + p * step] > 0.f) m = fmaxf(m, a.ws_m[base + p * step]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float l = 0.f;
      for (int p = lane; p < a.splits; p += 32) {
        const float lp = a.ws_l[base + p * step];
        if (lp > 0.f) l += lp * fast_exp2(a.ws_m[base + p * step] - m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) {
        s_m[r] = m == -INFINITY ? 0.f : m;
        s_inv[r] = l > 0.f ? 1.f / l : 0.f;  // a row that sees nothing has no weights
      }
    }
    __syncthreads();
    if (t < L) {
#pragma unroll 4
      for (int r = 0; r < n; ++r)
        share += fast_exp2(__ldcs(raw + (size_t)(r0 + r) * kTileTokens) - s_m[r]) * s_inv[r];
    }
  }
  if (t < L) ledger_write(a.scores, a.row_pos, a.seq_lens, seq, at, t, Lc, a.q_len, old, share);
}

template <typename T, int D, bool KV8>
cudaError_t launch_mass_t(const CUtensorMap &qmap, const LedgerArgs &a, cudaStream_t st) {
  auto kern = mass_tc_kernel<T, D, KV8>;
  static std::atomic<unsigned long long> opted{0};  // bit per device: smem opt-in done
  static std::atomic<int> sm_count[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(opted.load(std::memory_order_acquire) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             MassLayout<D>::smem_bytes(kMassMaxSeqs));
    if (e != cudaSuccess) return e;
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    sm_count[dev].store(sms, std::memory_order_relaxed);
    opted.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  const long long most = (long long)a.num_seqs * a.num_kv_heads * ((a.max_rows + kMassUnit - 1) / kMassUnit);
  if (most > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(most, sm_count[dev].load(std::memory_order_relaxed)), 1, 1);
  cfg.blockDim = dim3(kMassThreads, 1, 1);
  cfg.dynamicSmemBytes = MassLayout<D>::smem_bytes(a.num_seqs);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, qmap, a);
}

template <typename T>
cudaError_t mass_t(const CUtensorMap &qmap, const LedgerArgs &a, int head_dim, bool kv8, cudaStream_t s) {
  if (kv8) return launch_mass_t<T, 128, true>(qmap, a, s);
  if (head_dim == 128) return launch_mass_t<T, 128, false>(qmap, a, s);
  return launch_mass_t<T, 64, false>(qmap, a, s);
}

}  // namespace

cudaError_t launch_ledger(const LedgerArgs &a, cudaStream_t s) {
  const long long blocks = (long long)a.num_seqs * a.num_kv_heads *
                           ((a.max_rows + kLedgerThreads - 1) / kLedgerThreads);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(ledger_kernel, (unsigned)blocks, kLedgerThreads, s, a);
}

cudaError_t launch_mass(const CUtensorMap &qmap, const LedgerArgs &a, int head_dim, bool fp16,
                        bool kv8, cudaStream_t s) {
  return fp16 ? mass_t<__half>(qmap, a, head_dim, kv8, s)
              : mass_t<__nv_bfloat16>(qmap, a, head_dim, kv8, s);
}

void mass_q_box(int group, int *heads, int *tokens) {
  const MassGeo g = mass_geo(group);
  *heads = g.hb;
  *tokens = g.tb;
}

int mass_max_seqs() { return kMassMaxSeqs; }

}  // namespace pa
