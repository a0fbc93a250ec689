// pa_verify.cu -- verification of drafted tokens against the target's probabilities,
// from random numbers that the caller gives.
//
// For sequence i with drafts x_0 .. x_{m-1} (m = draft_lens[i]), target probabilities
// p_j, draft probabilities q_j and uniforms u_j: draft j is accepted while
//   u_j q_j(x_j) < p_j(x_j)                                  (all earlier ones accepted)
// With a = the number accepted, one more token is sampled from the weights
//   w(v) = max(p_a(v) - q_a(v), 0)   if a < m   (the residual distribution)
//   w(v) = p_m(v)                    if a = m
// as the first v with w(0) + .. + w(v) > s W, W the sum of all weights, s the
// sequence's sampling uniform.  The tokens then follow the target's distribution
// ("推理机制动态图解（进阶）" §3; "Scaling Book 入门第 11 章" §11.7: accept with
// min(1, p / q), else resample from (p - q)+).
//
// The answer is a token id, so sums decide at borders: with a vocabulary of 10^5
// tokens an fp32 sum of the weights (error ~1e-7 of the total) lands on the wrong side
// of one of the borders in about one call in a hundred.  The weights are therefore
// summed as fp32 pairs (value, rounding error; Knuth's two-sum) and reduced in fp64;
// u q < p is compared in fp64, where the product of two fp32 is exact.
//
// The fp64 rate of GB300 is two operations a clock and SM, so fp64 appears only where a
// warp reduces once.
//
// A sequence reads the drafted tokens' entries, then one vocabulary row of p and one
// of q.  One thread-block cluster per sequence: its CTAs sum a slice of the row each,
// exchange their sums through distributed shared memory, and the CTA whose slice
// holds the border searches it (the slice is in L2 by then): its CTAs' and warps' sums,
// then 1024 entries at a time through shared memory, so that the loads are coalesced and
// each lane still adds up 32 neighbours.
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 8;  // loads of each row in flight per thread
constexpr int kSearch = 1024;  // entries searched at once

struct VerifyArgs {
  int32_t *out_tokens, *num_accepted, *new_lens;
  const int32_t *context_lens;
  const float *target, *draft;
  const int32_t *draft_tokens, *draft_lens;
  const float *accept_u, *sample_u;
  int64_t p_row, p_seq, q_row, q_seq;  // elements between rows, between sequences
  int max_draft, vocab;
  unsigned *err;
};

// (s, c) += x: s the running fp32 sum, c the rounding errors it has dropped.
__device__ __forceinline__ void two_sum(float &s, float &c, float x) {
  const float t = __fadd_rn(s, x);
  const float z = __fsub_rn(t, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

// A weight as value + error: p - q split exactly, zero where it is not positive (or
// not finite).
struct Weight {
  float d, e;
};
__device__ __forceinline__ Weight weight_of(float p, float q) {
  Weight w;
  w.d = __fsub_rn(p, q);
  const float z = __fsub_rn(w.d, p);
  w.e = __fsub_rn(__fsub_rn(p, __fsub_rn(w.d, z)), __fadd_rn(q, z));
  if (!(w.d > 0.f && w.d <= 3.4028234e38f)) w.d = w.e = 0.f;
  return w;
}

// The weights of vocabulary row `p` (and `q`; skip: an entry whose weight is zero).
struct Row {
  const float *p, *q;
  int skip;
  __device__ __forceinline__ Weight at(int v) const {
    if (v == skip) return Weight{0.f, 0.f};
    return weight_of(__ldg(p + v), q ? __ldg(q + v) : 0.f);
  }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ double warp_scan(double x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Among 32 consecutive parts of sum x (one per lane), base the sum before them: the
// first whose running sum exceeds `border`, else the last with x > 0 (rounding at the
// end of the row), else -1.  *before = the running sum before it.
__device__ __forceinline__ int find_part(double x, double base, double border, double *before) {
  const double incl = base + warp_scan(x);
  const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && incl > border);
  const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
  const int k = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
  const double prev = __shfl_sync(0xffffffffu, incl - x, k < 0 ? 0 : k);
  *before = prev;
  return k;
}

__device__ __forceinline__ double dsmem_ld_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

// fp32 pair sum of the weights of entries [lo, hi), lane by lane (lo + lane, + 32, ...).
template <bool Q>
__device__ __forceinline__ void sum_range(const Row &row, int lo, int hi, float &s, float &c) {
  const int lane = threadIdx.x & 31;
  int v = lo + lane;
  for (; v + 32 * (kUnroll - 1) < hi; v += 32 * kUnroll) {
    float p[kUnroll], q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      p[u] = __ldg(row.p + v + 32 * u);
      if (Q) q[u] = __ldg(row.q + v + 32 * u);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (Q) {
        const Weight w = weight_of(p[u], q[u]);
        two_sum(s, c, w.d);
        c += w.e;
      } else {
        two_sum(s, c, v + 32 * u == row.skip ? 0.f : weight_of(p[u], 0.f).d);
      }
    }
  }
  float p[kUnroll], q[kUnroll];  // the rest
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const bool in = v + 32 * u < hi;
    p[u] = in ? __ldg(row.p + v + 32 * u) : 0.f;
    q[u] = (Q && in) ? __ldg(row.q + v + 32 * u) : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    Weight w = weight_of(p[u], q[u]);
    if (v + 32 * u == row.skip) w.d = w.e = 0.f;
    two_sum(s, c, w.d);
    c += w.e;
  }
}

__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a) {
  __shared__ double warp_part[kWarps];
  __shared__ double cta_part;
  __shared__ Weight s_w[32 * 33];  // 1024 searched weights, 32 a row
  __shared__ int s_count, s_given, s_skip;
  pa::griddep_wait();
  pa::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int csize = (int)pa::cluster_nctarank(), crank = (int)pa::cluster_ctarank();
  const int seq = blockIdx.x / csize;
  const float *p0 = a.target + seq * a.p_seq;
  const float *q0 = a.draft ? a.draft + seq * a.q_seq : nullptr;
  const int32_t *x = a.draft_tokens + (int64_t)seq * a.max_draft;

  // acceptance: every CTA's first warp works it out
  if (warp == 0) {
    int given = a.draft_lens ? __ldg(a.draft_lens + seq) : a.max_draft;
    if (given < 0 || given > a.max_draft) {
      if (lane == 0 && crank == 0) pa::record_error(a.err, pa::kErrCheck);
      given = min(max(given, 0), a.max_draft);
    }
    int count = given;
    for (int j0 = 0; j0 < given; j0 += 32) {
      const int j = j0 + lane;
      bool ok = true;
      if (j < given) {
        const int tok = __ldg(x + j);
        if (tok < 0 || tok >= a.vocab) {
          if (crank == 0) pa::record_error(a.err, pa::kErrCheck);
          ok = false;
        } else {
          const double p = __ldg(p0 + j * a.p_row + tok);
          const double q = q0 ? (double)__ldg(q0 + j * a.q_row + tok) : 1.0;
          ok = (double)__ldg(a.accept_u + (int64_t)seq * a.max_draft + j) * q < p;
        }
      }
      const unsigned bad = ~__ballot_sync(0xffffffffu, ok);
      if (bad) {
        count = j0 + __ffs(bad) - 1;
        break;
      }
    }
    if (lane == 0) {
      s_count = count;
      s_given = given;
      // without draft probabilities q is 1 at the draft: only its weight vanishes
      s_skip = (count < given && !q0) ? __ldg(x + count) : -1;
    }
  }
  __syncthreads();
  const int count = s_count, given = s_given;
  Row row;
  row.p = p0 + count * a.p_row;
  row.q = (count < given && q0) ? q0 + count * a.q_row : nullptr;
  row.skip = s_skip;

  // slice of this CTA, ranges of its warps: whole multiples of 32 entries
  const int per_warp = ((a.vocab + csize * kWarps - 1) / (csize * kWarps) + 31) & ~31;
  int token = -1;
  // round 0: the weights above; round 1 (their sum is zero: the distributions agree to
  // rounding, or the row is empty): the target row itself
  for (int round = 0; round < 2; ++round) {
    const int64_t lo64 = (int64_t)(crank * kWarps + warp) * per_warp;
    const int lo = (int)min((int64_t)a.vocab, lo64), hi = (int)min((int64_t)a.vocab, lo64 + per_warp);
    float s = 0.f, c = 0.f;
    if (row.q)
      sum_range<true>(row, lo, hi, s, c);
    else
      sum_range<false>(row, lo, hi, s, c);
    const double part = warp_sum((double)s + (double)c);
    if (lane == 0) warp_part[warp] = part;
    __syncthreads();
    if (warp == 0) {
      const double all = warp_sum(lane < kWarps ? warp_part[lane] : 0.0);
      if (lane == 0) cta_part = all;
    }
    pa::cluster_sync_all();
    if (warp == 0) {
      // every CTA finds the CTA whose slice holds the border; that one goes on
      const double mine = lane < csize ? dsmem_ld_f64(pa::dsmem_map(pa::smem_u32(&cta_part), lane)) : 0.0;
      const double total = warp_sum(mine);
      const double border = (double)__ldg(a.sample_u + seq) * total;
      double before;
      const int who = find_part(mine, 0.0, border, &before);
      if (who == crank) {
        const int w = find_part(lane < kWarps ? warp_part[lane] : 0.0, before, border, &before);
        if (w >= 0) {
          const int64_t l64 = (int64_t)(crank * kWarps + w) * per_warp;
          const int wlo = (int)min((int64_t)a.vocab, l64);
          const int whi = (int)min((int64_t)a.vocab, l64 + per_warp);
          for (int g0 = wlo; g0 < whi; g0 += kSearch) {
            const int g1 = min(whi, g0 + kSearch);
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {
              const int v = g0 + 32 * j + lane;
              s_w[33 * j + lane] = v < g1 ? row.at(v) : Weight{0.f, 0.f};
            }
            __syncwarp();
            float ls = 0.f, lc = 0.f;  // entries [g0 + 32 lane, + 32)
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {
              const Weight x = s_w[33 * lane + j];
              two_sum(ls, lc, x.d);
              lc += x.e;
            }
            const double sum = (double)ls + (double)lc;
            const double base = before;
            double at;
            const int part = find_part(sum, base, border, &at);
            if (part >= 0) {
              const Weight x = s_w[33 * part + lane];
              const int e = find_part((double)x.d + (double)x.e, at, border, &at);
              if (e >= 0) token = g0 + 32 * part + e;
            }
            before = base + warp_sum(sum);
            __syncwarp();
            if (before > border) break;  // else the border lies further on, or in rounding
          }
        }
      }
      const bool none = who < 0 && round == 1;  // no weight anywhere: no token
      if (who == crank || (none && crank == 0)) {
        int32_t *out = a.out_tokens + (int64_t)seq * (a.max_draft + 1);
        for (int j = lane; j <= a.max_draft; j += 32)
          out[j] = j < count ? __ldg(x + j) : j == count ? token : -1;
        if (lane == 0) {
          if (none) pa::record_error(a.err, pa::kErrCheck);
          a.num_accepted[seq] = count;
          if (a.new_lens)
            a.new_lens[seq] = max(0, __ldg(a.context_lens + seq) - (a.max_draft - count));
        }
      }
      if (lane == 0) s_given = who;
    }
    pa::cluster_sync_all();  // the sums have been read: they may be written again, or the CTA exit
    if (s_given >= 0) break;
    row.q = nullptr;
    row.skip = -1;
  }
}

}  // namespace

extern "C" PA_API pa_status pa_verify_drafts(
    int32_t *out_tokens, int32_t *num_accepted, int32_t *new_lens, const int32_t *context_lens,
    const float *target_probs, const float *draft_probs, const int32_t *draft_tokens,
    const int32_t *draft_lens, const float *accept_u, const float *sample_u, int num_seqs,
    int max_draft, int vocab, int64_t target_stride, int64_t draft_stride, void *stream) {
  if (!out_tokens || !num_accepted || !target_probs || !draft_tokens || !accept_u || !sample_u)
    return PA_ERR_INVALID_ARG;
  if (new_lens && !context_lens) return PA_ERR_INVALID_ARG;
  if (num_seqs <= 0 || max_draft <= 0 || vocab <= 0 || vocab > (1 << 30)) return PA_ERR_INVALID_ARG;
  if (target_stride < vocab || (draft_probs && draft_stride < vocab)) return PA_ERR_INVALID_ARG;
  if (target_stride > ((int64_t)1 << 40) || draft_stride > ((int64_t)1 << 40))
    return PA_ERR_INVALID_ARG;
  if (max_draft > 4095) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_seqs * (max_draft + 1) >= (int64_t)1 << 31) return PA_ERR_INVALID_ARG;
  const void *ptrs[10] = {out_tokens,   num_accepted, new_lens,   context_lens, target_probs,
                          draft_probs,  draft_tokens, draft_lens, accept_u,     sample_u};
  for (const void *p : ptrs)
    if (!pa::aligned4(p)) return PA_ERR_INVALID_ARG;
  VerifyArgs a;
  a.out_tokens = out_tokens;
  a.num_accepted = num_accepted;
  a.new_lens = new_lens;
  a.context_lens = context_lens;
  a.target = target_probs;
  a.draft = draft_probs;
  a.draft_tokens = draft_tokens;
  a.draft_lens = draft_lens;
  a.accept_u = accept_u;
  a.sample_u = sample_u;
  a.p_row = target_stride;
  a.p_seq = target_stride * (max_draft + 1);
  a.q_row = draft_stride;
  a.q_seq = draft_stride * max_draft;
  a.max_draft = max_draft;
  a.vocab = vocab;
  a.err = pa::error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  const int cluster = 8;
  if ((int64_t)num_seqs * cluster >= (int64_t)1 << 31) return PA_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_seqs * cluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
