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
//     KV head's rows (pa_decode.cuh), else by finish_kernel;
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
constexpr int kLedgerRows = 4 * kLedgerThreads;  // cached rows of a CTA, four a thread
constexpr int kRowBatch = 64;   // query rows whose statistics are in shared memory at once
constexpr int kAhead = 4;       // scores loaded before the statistics are known

// What follows the decode pass when its CTAs do not hold a KV head's row sums: CTAs below
// combine_blocks merge the partitions into the output (SPREAD: one dimension per lane),
// the others take kLedgerRows cached rows of one (sequence, KV head) each.  One launch
// for both: neither is long (6.6 and 20 us as two launches over 4 x 32768 tokens in 16
// partitions), and both wait on loads.
template <typename T, int D, bool SPREAD>
__global__ void __launch_bounds__(kLedgerThreads) finish_kernel(const LedgerArgs a, const CombineArgs c,
                                                                int combine_blocks) {
  __shared__ float s_m[kRowBatch], s_inv[kRowBatch];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x < combine_blocks) {
    constexpr int kParts = SPREAD ? D / 32 : 1;
    const int gw = blockIdx.x * (kLedgerThreads / 32) + warp;
    if (gw / kParts >= c.num_seqs * c.rows_per_seq) return;
    if constexpr (SPREAD)
      combine_row_part<T, D>(c, gw / kParts, gw % kParts);
    else
      combine_row<T, D>(c, gw);
    return;
  }
  const int id = blockIdx.x - combine_blocks;
  const int chunks = (a.max_rows + kLedgerRows - 1) / kLedgerRows;
  const int unit = id / chunks, chunk = id % chunks;
  const int seq = unit / a.num_kv_heads, kvh = unit % a.num_kv_heads;
  const int Lc = max(0, __ldg(a.context_lens + seq)), L = min(Lc, a.max_rows);
  if (chunk * kLedgerRows >= L) return;
  // this thread's four cached rows: slots 4 i .. 4 i + 3 of a tile
  const int tile = chunk * (kLedgerRows / kTileTokens) + threadIdx.x / 4;
  const int slot = 4 * (threadIdx.x % 4);
  const float4 *raw = reinterpret_cast<const float4 *>(
      a.raw_scores + ((size_t)unit * a.max_tiles + tile) * a.rows * kTileTokens + slot);
  constexpr int kStep = kTileTokens / 4;  // float4s between query rows
  const int64_t led = (int64_t)unit * a.max_rows;
  int t[4];
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = tile * kTileTokens + score_token(a.rows, slot + i);
    o[i] = t[i] < L ? a.scores[led + t[i]] : 0.f;
  }
  const bool in = tile * kTileTokens < L;
  float4 x[kAhead];
#pragma unroll
  for (int r = 0; r < kAhead; ++r) {
    x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in && r < a.rows) x[r] = raw[r * kStep];
  }
  const int heads = a.group * a.num_kv_heads;
  float4 share = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r0 = 0; r0 < a.rows; r0 += kRowBatch) {
    const int n = min(kRowBatch, a.rows - r0);
    __syncthreads();
    for (int r = warp; r < n; r += kLedgerThreads / 32) {
      // a warp merges the partitions' statistics of query token u, head h
      const int u = (r0 + r) / a.group, h = kvh * a.group + (r0 + r) % a.group;
      const size_t base = (size_t)seq * a.splits * a.q_len * heads + (size_t)u * heads + h;
      const size_t step = (size_t)a.q_len * heads;
      float m = -INFINITY, l = 0.f;
      for (int p0 = 0; p0 < a.splits; p0 += 32) {
        const int p = p0 + lane;
        const float lp = p < a.splits ? a.ws_l[base + p * step] : 0.f;
        const float mp = p < a.splits ? a.ws_m[base + p * step] : -INFINITY;
        float mx = lp > 0.f ? mp : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(mx, m);
        if (mx == -INFINITY) continue;
        l = l * fast_exp2(m - mx) + (lp > 0.f ? lp * fast_exp2(mp - mx) : 0.f);
        m = mx;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) {
        s_m[r] = m == -INFINITY ? 0.f : m;
        s_inv[r] = l > 0.f ? 1.f / l : 0.f;  // a row that sees nothing has no weights
      }
    }
    __syncthreads();
    auto add = [&](const float4 &v, int r) {
      const float m = s_m[r], inv = s_inv[r];
      share.x += fast_exp2(v.x - m) * inv;
      share.y += fast_exp2(v.y - m) * inv;
      share.z += fast_exp2(v.z - m) * inv;
      share.w += fast_exp2(v.w - m) * inv;
    };
    int r = 0;
    if (r0 == 0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < n) add(x[i], i);
      r = kAhead;
    }
    if (in) {
#pragma unroll 4
      for (; r < n; ++r) add(raw[(size_t)(r0 + r) * kStep], r);
    }
  }
  const float s[4] = {share.x, share.y, share.z, share.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t[i] < L)
      ledger_write(a.scores, a.row_pos, a.seq_lens, seq, led + t[i], t[i], Lc, a.q_len, o[i], s[i]);
}

template <typename T, int D>
cudaError_t finish_t(const LedgerArgs &a, const CombineArgs &c, bool combine, cudaStream_t st) {
  const long long ledger = (long long)a.num_seqs * a.num_kv_heads * ((a.max_rows + kLedgerRows - 1) / kLedgerRows);
  const long long rows = combine ? (long long)c.num_seqs * c.rows_per_seq : 0;
  const bool spread = combine && combine_spread(c.num_splits, rows);
  const long long warps = spread ? rows * (D / 32) : rows;
  const long long blocks = (warps + kLedgerThreads / 32 - 1) / (kLedgerThreads / 32);
  if (ledger + blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(ledger + blocks), 1, 1);
  return spread ? launch_dependent(finish_kernel<T, D, true>, grid, kLedgerThreads, st, a, c, (int)blocks)
                : launch_dependent(finish_kernel<T, D, false>, grid, kLedgerThreads, st, a, c, (int)blocks);
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

cudaError_t launch_finish(const LedgerArgs &a, const CombineArgs *c, int head_dim, bool fp16,
                          cudaStream_t s) {
  const CombineArgs cc = c ? *c : CombineArgs();
  if (head_dim == 128)
    return fp16 ? finish_t<__half, 128>(a, cc, c != nullptr, s)
                : finish_t<__nv_bfloat16, 128>(a, cc, c != nullptr, s);
  return fp16 ? finish_t<__half, 64>(a, cc, c != nullptr, s)
              : finish_t<__nv_bfloat16, 64>(a, cc, c != nullptr, s);
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
