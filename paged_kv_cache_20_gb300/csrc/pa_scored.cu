// pa_scored.cu -- the ledger of accumulated attention weight: what each cached row
// drew from this step's queries, added to the row's score.
//
// For KV head h of sequence i and cached row t
//   share(t) = sum over the head's query rows r that see t of
//              2^(s_rt - m_r) / l_r                 (s in base-2 units)
// with m_r and l_r the row's softmax maximum and sum.  These are known only after the
// attention pass, so the weights take a second look at the scores:
//   * up to 16 query tokens: the decode pass leaves its scores in the workspace
//     (ledger_kernel reads them back: 4 bytes per row and head against the 2 head_dim
//     16-bit values per row of reading K again and V);
//   * more: the scores would outgrow the cache, so mass_kernel computes them again
//     from K and q.
// Rows that this step appended (the last q_len) start their scores here, and their
// positions are noted; a row's score is written by one thread, so the sums have one
// order.
#include <cuda_runtime.h>

#include "pa_decode.cuh"
#include "pa_launch.h"
#include "pa_scored.h"

namespace pa {

namespace {

constexpr int kLedgerThreads = 256;
constexpr int kRowBatch = 256;  // rows whose statistics are in shared memory at once

// Score and position of cached row t (Lc: the context length as given, which may
// exceed the table).
__device__ __forceinline__ void ledger_write(const LedgerArgs &a, int seq, int64_t at, int t, int Lc,
                                             float share) {
  const bool fresh = t >= Lc - a.q_len;
  a.scores[at] = fresh ? share : a.scores[at] + share;
  if (fresh && a.row_pos) a.row_pos[at] = __ldg(a.seq_lens + seq) - Lc + t;
}

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
  for (int r0 = 0; r0 < a.rows; r0 += kRowBatch) {
    const int n = min(kRowBatch, a.rows - r0);
    __syncthreads();
    for (int r = threadIdx.x; r < n; r += kLedgerThreads) {
      // merge the partitions' statistics of query token u, head h
      const int u = (r0 + r) / a.group, h = kvh * a.group + (r0 + r) % a.group;
      const size_t base = (size_t)seq * a.splits * a.q_len * heads + (size_t)u * heads + h;
      float m = -INFINITY, l = 0.f;
      for (int p = 0; p < a.splits; ++p) {
        const float mp = a.ws_m[base + (size_t)p * a.q_len * heads];
        const float lp = a.ws_l[base + (size_t)p * a.q_len * heads];
        if (!(lp > 0.f)) continue;
        const float mn = fmaxf(m, mp);
        l = l * fast_exp2(m - mn) + lp * fast_exp2(mp - mn);
        m = mn;
      }
      s_m[r] = m == -INFINITY ? 0.f : m;
      s_inv[r] = l > 0.f ? 1.f / l : 0.f;  // a row that sees nothing has no weights
    }
    __syncthreads();
    if (t < L)
      for (int r = 0; r < n; ++r)
        share += fast_exp2(raw[(size_t)(r0 + r) * kTileTokens] - s_m[r]) * s_inv[r];
  }
  if (t < L) ledger_write(a, seq, (int64_t)unit * a.max_rows + t, t, Lc, share);
}

// Element (two of them) of a cached row as the MMA operand of type T: 16-bit as it
// is, e4m3 widened (exact in fp16 and bf16).
template <typename T, bool KV8>
__device__ __forceinline__ uint32_t load_pair(const void *cache, int64_t at) {
  if constexpr (KV8) {
    const uint32_t h2 = e4m3x2_to_f16x2(__ldg(reinterpret_cast<const uint16_t *>(
        static_cast<const uint8_t *>(cache) + at)));
    const float2 f = Elt<__half>::to_f2(h2);
    return Elt<T>::from_f2(f.x, f.y);
  } else {
    return __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(cache) + at));
  }
}

// Many query rows: S^T = K q^T again, 16 cached rows a warp (the MMA's M, its K
// fragments in registers) by 8 query rows at a time.
template <typename T, int D, bool KV8>
__global__ void __launch_bounds__(256) mass_kernel(const LedgerArgs a) {
  constexpr int KS = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int groups = (a.max_tiles + 7) / 8;
  const int unit = blockIdx.x / groups, tile = (blockIdx.x % groups) * 8 + warp;
  const int seq = unit / a.num_kv_heads, kvh = unit % a.num_kv_heads;
  const int Lc = max(0, __ldg(a.context_lens + seq)), L = min(Lc, a.max_rows);
  const int t0 = tile * kTileTokens;
  if (t0 >= L) return;
  const int heads = a.group * a.num_kv_heads;
  uint32_t ka[KS][4];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int t = t0 + g + 8 * hh;
    int64_t row = -1;
    if (t < L) {
      const int id = __ldg(a.block_tables + (size_t)seq * a.max_blocks_per_seq + t / a.block_size);
      if (id >= 0 && id < a.num_blocks)  // (a bad id reads as zeros; the attention pass reports it)
        row = (((int64_t)id * a.num_kv_heads + kvh) * a.block_size + t % a.block_size) * D;
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      ka[ks][hh] = row < 0 ? 0u : load_pair<T, KV8>(a.k_cache, row + ks * 16 + 2 * c);
      ka[ks][hh + 2] = row < 0 ? 0u : load_pair<T, KV8>(a.k_cache, row + ks * 16 + 2 * c + 8);
    }
  }
  const float scale = a.scale_log2 * (KV8 ? __ldg(a.k_scale + kvh) : 1.f);
  // query tokens before u0 see none of these rows
  const int u0 = max(0, t0 - (Lc - a.q_len));
  float share[2] = {0.f, 0.f};
  for (int r0 = u0 * a.group; r0 < a.rows; r0 += 8) {
    const int rq = r0 + g;  // the query row whose elements this lane loads
    const int uq = rq / a.group, hq = kvh * a.group + rq % a.group;
    const T *q = static_cast<const T *>(a.q) + ((size_t)(seq * a.q_len + uq) * heads + hq) * D;
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t b0 = 0u, b1 = 0u;
      if (rq < a.rows) {
        b0 = __ldg(reinterpret_cast<const uint32_t *>(q + ks * 16 + 2 * c));
        b1 = __ldg(reinterpret_cast<const uint32_t *>(q + ks * 16 + 2 * c + 8));
      }
      Elt<T>::mma16816(sc, ka[ks], b0, b1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 2 * c + (i & 1), t = t0 + g + 8 * (i >> 1);
      if (r >= a.rows) continue;
      const int u = r / a.group;
      if (t > Lc - a.q_len + u) continue;
      const size_t row = (size_t)(seq * a.q_len + u) * heads + kvh * a.group + r % a.group;
      const float l = a.ws_l[row];
      share[i >> 1] += l > 0.f ? fast_exp2(sc[i] * scale - a.ws_m[row]) / l : 0.f;
    }
  }
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    share[hh] += __shfl_xor_sync(0xffffffffu, share[hh], 1);
    share[hh] += __shfl_xor_sync(0xffffffffu, share[hh], 2);
    const int t = t0 + g + 8 * hh;
    if (c == 0 && t < L) ledger_write(a, seq, (int64_t)unit * a.max_rows + t, t, Lc, share[hh]);
  }
}

template <typename T>
cudaError_t mass_t(const LedgerArgs &a, int head_dim, bool kv8, unsigned blocks, cudaStream_t s) {
  if (kv8) return launch_dependent(mass_kernel<T, 128, true>, blocks, 256, s, a);
  if (head_dim == 128) return launch_dependent(mass_kernel<T, 128, false>, blocks, 256, s, a);
  return launch_dependent(mass_kernel<T, 64, false>, blocks, 256, s, a);
}

}  // namespace

cudaError_t launch_ledger(const LedgerArgs &a, cudaStream_t s) {
  const long long blocks = (long long)a.num_seqs * a.num_kv_heads *
                           ((a.max_rows + kLedgerThreads - 1) / kLedgerThreads);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(ledger_kernel, (unsigned)blocks, kLedgerThreads, s, a);
}

cudaError_t launch_mass(const LedgerArgs &a, int head_dim, bool fp16, bool kv8, cudaStream_t s) {
  const long long blocks = (long long)a.num_seqs * a.num_kv_heads * ((a.max_tiles + 7) / 8);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return fp16 ? mass_t<__half>(a, head_dim, kv8, (unsigned)blocks, s)
              : mass_t<__nv_bfloat16>(a, head_dim, kv8, (unsigned)blocks, s);
}

}  // namespace pa
