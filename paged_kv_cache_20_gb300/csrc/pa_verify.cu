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
// of one of the borders in about one call in a hundred.  All sums here are pairs of
// fp32 (the rounded sum and the rounding errors it dropped, by Knuth's two-sum, themselves
// added in fp32), good to about 2^-46 of the total (2^-47.2 the worst of 40 rows of 32000 and
// 131071 entries, the same additions redone on the CPU); a uniform that falls so near a border may take either
// token.  The fp64 rate of GB300 is two operations a clock and SM
// (scans in fp64 made the search 17 us of 35 in a batch of 64).  u q < p is compared in
// fp64, where the product of two fp32 is exact.
//
// A sequence reads the drafted tokens' entries, then one vocabulary row of p and one
// of q.  One thread-block cluster per sequence: its CTAs sum a slice of the row each,
// exchange their sums through distributed shared memory, and the CTA whose slice
// holds the border searches it (the slice is in L2 by then): by its warps' ranges, then
// 2048 entries at a time with 256 a warp, each lane's eight loads in flight at once.
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 8;  // loads of each row in flight per thread
constexpr int kCluster = 8;
constexpr int kPiece = 32 * kUnroll;        // entries a warp searches at once
constexpr int kSearch = kWarps * kPiece;    // and the CTA

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

// s the rounded sum, c the rounding errors it has dropped.
struct Pair {
  float s, c;
  __device__ __forceinline__ bool positive() const { return s > 0.f; }  // (weights are >= 0)
};

__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair r;
  r.s = __fadd_rn(a.s, b.s);
  const float z = __fsub_rn(r.s, a.s);
  r.c = __fadd_rn(__fadd_rn(a.c, b.c), __fadd_rn(__fsub_rn(a.s, __fsub_rn(r.s, z)), __fsub_rn(b.s, z)));
  return r;
}

// a > b: where the rounded sums are close their difference is exact
__device__ __forceinline__ bool greater(Pair a, Pair b) {
  return __fadd_rn(__fsub_rn(a.s, b.s), __fsub_rn(a.c, b.c)) > 0.f;
}

// u * a
__device__ __forceinline__ Pair scaled(float u, Pair a) {
  Pair r;
  r.s = __fmul_rn(u, a.s);
  r.c = __fadd_rn(__fmaf_rn(u, a.s, -r.s), __fmul_rn(u, a.c));
  return r;
}

__device__ __forceinline__ Pair shfl(Pair a, int lane) {
  return Pair{__shfl_sync(0xffffffffu, a.s, lane), __shfl_sync(0xffffffffu, a.c, lane)};
}

// Sum over groups of N lanes.
template <int N>
__device__ __forceinline__ Pair group_sum(Pair x) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1)
    x = add(x, Pair{__shfl_xor_sync(0xffffffffu, x.s, o), __shfl_xor_sync(0xffffffffu, x.c, o)});
  return x;
}

// A weight: p - q split exactly into value and error, zero where it is not positive (or
// not finite).
__device__ __forceinline__ Pair weight_of(float p, float q) {
  Pair w;
  w.s = __fsub_rn(p, q);
  const float z = __fsub_rn(w.s, p);
  w.c = __fsub_rn(__fsub_rn(p, __fsub_rn(w.s, z)), __fadd_rn(q, z));
  if (!(w.s > 0.f && w.s <= 3.4028234e38f)) w.s = w.c = 0.f;
  return w;
}

// The weights of vocabulary row `p` (and `q`; skip: an entry whose weight is zero).
struct Row {
  const float *p, *q;
  int skip;
};

// Among the parts x of lanes 0 .. N-1 (in order; other lanes hold zeros), `base` the sum
// before them: the first part whose running sum exceeds `border`, else the last positive
// one (rounding at the end of the row), else -1.  *before = the running sum before it,
// *over = whether the border was exceeded.
template <int N>
__device__ __forceinline__ int find_part(Pair x, Pair base, Pair border, Pair *before, bool *over) {
  const int lane = threadIdx.x & 31;
  Pair incl = x;
#pragma unroll
  for (int o = 1; o < N; o <<= 1) {
    const Pair y = {__shfl_up_sync(0xffffffffu, incl.s, o), __shfl_up_sync(0xffffffffu, incl.c, o)};
    if (lane >= o) incl = add(y, incl);
  }
  incl = add(base, incl);
  const unsigned past = __ballot_sync(0xffffffffu, lane < N && x.positive() && greater(incl, border));
  const unsigned some = __ballot_sync(0xffffffffu, lane < N && x.positive());
  const int k = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : -1;
  *over = past != 0u;
  const Pair prev = shfl(incl, k > 0 ? k - 1 : 0);
  *before = k > 0 ? prev : base;
  return k;
}

// fp32 pair sum of the weights of this lane's entries of [lo, hi): lo + lane, + 32, ...
template <bool Q>
__device__ __forceinline__ Pair sum_range(const Row &row, int lo, int hi) {
  const int lane = threadIdx.x & 31;
  Pair sum = {0.f, 0.f};
  int v = lo + lane;
  for (; v + 32 * (kUnroll - 1) < hi; v += kPiece) {
    float p[kUnroll], q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      p[u] = __ldg(row.p + v + 32 * u);
      if (Q) q[u] = __ldg(row.q + v + 32 * u);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      Pair w = weight_of(p[u], Q ? q[u] : 0.f);
      if (!Q && v + 32 * u == row.skip) w = Pair{0.f, 0.f};
      sum = add(sum, w);
    }
  }
  for (; v < hi; v += 32) {
    Pair w = weight_of(__ldg(row.p + v), Q ? __ldg(row.q + v) : 0.f);
    if (v == row.skip) w = Pair{0.f, 0.f};
    sum = add(sum, w);
  }
  return sum;
}

__device__ __forceinline__ Pair dsmem_ld_pair(uint32_t addr) {
  return Pair{pa::dsmem_ld_f32(addr), pa::dsmem_ld_f32(addr + 4)};
}

__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a) {
  __shared__ Pair warp_part[kWarps], piece_part[kWarps];
  __shared__ Pair cta_part;
  __shared__ int s_count, s_given, s_skip, s_token;
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
  // round 0: the weights above; round 1 (their sum is zero: the distributions agree to
  // rounding, or the row is empty): the target row itself
  for (int round = 0; round < 2; ++round) {
    const int64_t lo64 = (int64_t)(crank * kWarps + warp) * per_warp;
    const int lo = (int)min((int64_t)a.vocab, lo64), hi = (int)min((int64_t)a.vocab, lo64 + per_warp);
    const Pair part = group_sum<32>(row.q ? sum_range<true>(row, lo, hi) : sum_range<false>(row, lo, hi));
    if (lane == 0) warp_part[warp] = part;
    __syncthreads();
    const Pair none = {0.f, 0.f};
    const Pair parts = lane < kWarps ? warp_part[lane] : none;
    if (warp == 0) {
      const Pair all = group_sum<kWarps>(parts);
      if (lane == 0) {
        cta_part = all;
        s_token = -1;
      }
    }
    pa::cluster_sync_all();
    // every warp of every CTA finds the CTA whose slice holds the border
    const Pair slices = lane < csize ? dsmem_ld_pair(pa::dsmem_map(pa::smem_u32(&cta_part), lane)) : none;
    const Pair border = scaled(__ldg(a.sample_u + seq), shfl(group_sum<kCluster>(slices), 0));
    Pair before;
    bool over;
    const int who = find_part<kCluster>(slices, none, border, &before, &over);
    if (who == crank) {
      const int w = find_part<kWarps>(parts, before, border, &before, &over);
      const int64_t l64 = (int64_t)(crank * kWarps + w) * per_warp;
      const int wlo = (int)min((int64_t)a.vocab, l64), whi = (int)min((int64_t)a.vocab, l64 + per_warp);
      over = false;
      for (int g0 = wlo; g0 < whi && !over; g0 += kSearch) {
        // each warp weighs its piece of 256 entries, entry 32 j + lane in register j
        const int v0 = g0 + warp * kPiece + lane;
        float p[kUnroll], q[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const bool in = v0 + 32 * j < whi;
          p[j] = in ? __ldg(row.p + v0 + 32 * j) : 0.f;
          q[j] = (in && row.q) ? __ldg(row.q + v0 + 32 * j) : 0.f;
        }
        Pair x[kUnroll], sum = none;
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          x[j] = weight_of(p[j], q[j]);
          if (v0 + 32 * j == row.skip) x[j] = none;
          sum = add(sum, x[j]);
        }
        sum = group_sum<32>(sum);
        if (lane == 0) piece_part[warp] = sum;
        __syncthreads();
        const Pair pieces = lane < kWarps ? piece_part[lane] : none;
        const Pair all = add(before, shfl(group_sum<kWarps>(pieces), 0));
        Pair at;
        const int piece = find_part<kWarps>(pieces, before, border, &at, &over);
        if (piece == warp) {
          // its eight rows of 32 entries: their sums (lane j keeps row j's), then the entry
          Pair rows = none;
#pragma unroll
          for (int j = 0; j < kUnroll; ++j) {
            const Pair r = group_sum<32>(x[j]);
            if (lane == j) rows = r;
          }
          bool o;
          const int j = find_part<kUnroll>(rows, at, border, &at, &o);
          Pair mine = none;
#pragma unroll
          for (int i = 0; i < kUnroll; ++i)
            if (i == j) mine = x[i];
          const int e = find_part<32>(mine, at, border, &at, &o);
          if (lane == 0 && e >= 0) s_token = g0 + piece * kPiece + 32 * j + e;
        }
        before = all;
        __syncthreads();  // (over is the same in every warp: the border is found, or further on)
      }
    }
    const bool empty = who < 0 && round == 1;  // no weight anywhere: no token
    if (warp == 0 && (who == crank || (empty && crank == 0))) {
      const int token = s_token;
      int32_t *out = a.out_tokens + (int64_t)seq * (a.max_draft + 1);
      for (int j = lane; j <= a.max_draft; j += 32)
        out[j] = j < count ? __ldg(x + j) : j == count ? token : -1;
      if (lane == 0) {
        if (empty) pa::record_error(a.err, pa::kErrCheck);
        a.num_accepted[seq] = count;
        if (a.new_lens)
          a.new_lens[seq] = max(0, __ldg(a.context_lens + seq) - (a.max_draft - count));
      }
    }
    pa::cluster_sync_all();  // the sums have been read: they may be written again, or the CTA exit
    if (who >= 0) break;
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
  // A sequence's thread blocks read its inputs before one of them writes its outputs, but
  // sequences have no order: an output lies on an input only where every sequence's part
  // lies on its own (and context_lens is read last).
  const size_t lens = (size_t)num_seqs * 4, drafts = lens * max_draft, tokens = lens + drafts;
  auto shared = [](const void *p, size_t p_bytes, const void *q, size_t q_bytes, bool same_is_fine) {
    return p && q && pa::overlap(p, p_bytes, q, q_bytes) && !(same_is_fine && p == q);
  };
  const int32_t *old_lens = new_lens ? context_lens : nullptr;
  if (shared(new_lens, lens, old_lens, lens, true) || shared(new_lens, lens, draft_lens, lens, true) ||
      shared(new_lens, lens, draft_tokens, drafts, false) ||
      shared(num_accepted, lens, draft_lens, lens, true) || shared(num_accepted, lens, old_lens, lens, false) ||
      shared(num_accepted, lens, draft_tokens, drafts, false) ||
      shared(out_tokens, tokens, draft_tokens, drafts, num_seqs == 1) ||
      shared(out_tokens, tokens, draft_lens, lens, false) || shared(out_tokens, tokens, old_lens, lens, false) ||
      shared(out_tokens, tokens, num_accepted, lens, false) ||
      shared(out_tokens, tokens, new_lens, lens, false) || shared(num_accepted, lens, new_lens, lens, false))
    return PA_ERR_INVALID_ARG;
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
  const int cluster = kCluster;
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
