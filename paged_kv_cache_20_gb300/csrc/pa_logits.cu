// pa_logits.cu -- penalties for repeated tokens, biases and grammar masks on a step's
// logits, and the probabilities that the verification of drafts takes.
//
// Of entry v in row j of a sequence, with count the times v stands in its outputs (the
// history past the prompt and the drafts before row j) and seen whether it stands there or
// in the prompt:
//   y = seen ? (x > 0 ? x / repetition : x * repetition) : x
//   y = y - count * frequency;  y = y - presence if count > 0;  y = y + its biases
//   y = -inf where the mask's bit is clear
//   p = softmax(y / temperature), or with temperature <= 0 one at the largest y
// each operation rounded to fp32 by itself, so that the largest y does not depend on how
// they are fused.
//
// Bound by memory: a row is read once and written once.  A cluster of up to 8 thread blocks
// holds one row in registers, each a slice of the vocabulary; a warp takes its part of the
// row against its own maximum, and one cluster barrier exchanges every warp's maximum and
// sum.  The counts of a slice stand in shared memory for all rows of the sequence, each
// draft added before the next row, beside one bit an entry that says whether anything was
// counted: the rows' elements read that bit, few of them a count.  A row of an odd
// vocabulary starts anywhere: a thread's eight elements are aligned to 16 bytes of the row,
// not to the slice, whose ragged ends go by single elements.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "../../include/pagedattn.h"
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace pa {
namespace {

// All threads of the cluster (a warp arrives as one).
__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  cluster_sync_all();
}

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxBias = 1024;
constexpr int kMaxVocab = 1 << 18;
constexpr unsigned kPrompt = 1u << 31, kBias = 1u << 30;  // flags above an entry's count

struct LogitArgs {
  void *out;
  const void *logits;
  const int32_t *history, *history_lens, *prompt_lens, *drafts, *bias_ids, *mask;
  const float *repetition, *presence, *frequency, *bias_values, *temperature;
  int num_seqs, rows, vocab, max_history, num_bias;
  int slice;      // entries of a thread block, a multiple of 32
  int row_groups;  // row groups of a sequence, each of its own cluster
  int64_t out_stride, logits_stride, mask_seq, mask_row;
  unsigned *err;
};

template <typename T> struct In;
template <> struct In<__half> {
  static __device__ __forceinline__ float to_f(uint16_t v) { return __half2float(__ushort_as_half(v)); }
};
template <> struct In<__nv_bfloat16> {
  static __device__ __forceinline__ float to_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
};

// Eight elements from a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elt<T>::to_f2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ float load1(const T *p) {
  if constexpr (sizeof(T) == 4)
    return *p;
  else
    return In<T>::to_f(*reinterpret_cast<const uint16_t *>(p));
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(Elt<T>::from_f2(x[0], x[1]), Elt<T>::from_f2(x[2], x[3]),
                                                    Elt<T>::from_f2(x[4], x[5]), Elt<T>::from_f2(x[6], x[7])));
  }
}
template <typename T>
__device__ __forceinline__ void store1(T *p, float x) {
  if constexpr (sizeof(T) == 4)
    *p = x;
  else
    *reinterpret_cast<uint16_t *>(p) = Elt<T>::from_f(x);
}

// 2^x, subnormal results to zero (a probability below 2^-126 of the warp's largest)
__device__ __forceinline__ float ex2_flush(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void dsmem_st_f32x2(uint32_t addr, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// Bits v0 .. v0 + 7 of a bit array of `words` words (bits outside: 0).
template <typename Load>
__device__ __forceinline__ unsigned bits8(int v0, int words, Load load) {
  const int w = v0 >> 5, s = v0 & 31;  // (v0 may be negative: w = -1)
  const unsigned a = w >= 0 && w < words ? load(w) : 0u;
  const unsigned b = s > 24 && w + 1 < words ? load(w + 1) : 0u;
  return __funnelshift_r(a, b, s) & 0xffu;
}

// VPT: groups of eight elements a thread holds.
template <typename T, int VPT, bool PROBS>
__global__ void __launch_bounds__(kThreads) adjust_logits_kernel(const LogitArgs a) {
  using O = typename std::conditional<PROBS, float, T>::type;
  extern __shared__ unsigned s_words[];  // counts [slice], then one bit an entry [slice / 32]
  __shared__ __align__(8) float2 s_stat[2][kMaxCluster * kWarps];
  __shared__ int s_bias_id[kMaxBias];
  __shared__ float s_bias_v[kMaxBias];
  __shared__ int s_bias_n;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int csize = (int)cluster_nctarank(), crank = (int)cluster_ctarank();
  const int unit = blockIdx.x / csize;
  const int seq = unit / a.row_groups, group = unit % a.row_groups;
  const int j0 = (int)((int64_t)a.rows * group / a.row_groups);
  const int j1 = (int)((int64_t)a.rows * (group + 1) / a.row_groups);
  const int lo = min(a.vocab, crank * a.slice), hi = min(a.vocab, lo + a.slice);
  unsigned *count = s_words, *touched = s_words + a.slice;
  const bool counted = a.history != nullptr || a.drafts != nullptr || a.num_bias > 0;

  auto touch = [&](int e) { atomicOr(touched + (e >> 5), 1u << (e & 31)); };
  if (counted) {
    for (int i = threadIdx.x; i < a.slice + a.slice / 32; i += kThreads) s_words[i] = 0u;
    __syncthreads();
    if (a.history != nullptr) {
      int n = __ldg(a.history_lens + seq);
      if ((n < 0 || n > a.max_history) && threadIdx.x == 0 && crank == 0) record_error(a.err, kErrCheck);
      n = min(max(n, 0), a.max_history);
      const int prompt = a.prompt_lens ? __ldg(a.prompt_lens + seq) : 0;
      const int32_t *ids = a.history + (int64_t)seq * a.max_history;
#pragma unroll 4
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const int v = __ldg(ids + i);
        if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
        if (v >= lo && v < hi) {
          if (i < prompt)
            atomicOr(count + (v - lo), kPrompt);
          else
            atomicAdd(count + (v - lo), 1u);
          touch(v - lo);
        }
      }
    }
    if (a.drafts != nullptr)
      for (int i = threadIdx.x; i < j0; i += kThreads) {
        const int v = __ldg(a.drafts + (int64_t)seq * (a.rows - 1) + i);
        if (v >= lo && v < hi) {
          atomicAdd(count + (v - lo), 1u);
          touch(v - lo);
        }
      }
    // the slice's biases, in the list's order
    if (warp == 0) {
      int n = 0;
      for (int i0 = 0; i0 < a.num_bias; i0 += 32) {
        const int i = i0 + lane;
        const int v = i < a.num_bias ? __ldg(a.bias_ids + (int64_t)seq * a.num_bias + i) : -1;
        if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
        const bool mine = v >= lo && v < hi;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (mine) {
          const int at = n + __popc(who & ((1u << lane) - 1u));
          s_bias_id[at] = v - lo;
          s_bias_v[at] = __ldg(a.bias_values + (int64_t)seq * a.num_bias + i);
          atomicOr(count + (v - lo), kBias);
          touch(v - lo);
        }
        n += __popc(who);
      }
      if (lane == 0) s_bias_n = n;
    }
    __syncthreads();
  }
  const float rep = a.repetition ? __ldg(a.repetition + seq) : 1.f;
  const float pres = a.presence ? __ldg(a.presence + seq) : 0.f;
  const float freq = a.frequency ? __ldg(a.frequency + seq) : 0.f;
  const float temp = a.temperature ? __ldg(a.temperature + seq) : 1.f;
  const bool greedy = PROBS && !(temp > 0.f);
  // the exponent's factor; kept finite and above zero, so that -inf stays -inf
  const float fac = fminf(fmaxf(1.4426950408889634f / temp, 1e-38f), FLT_MAX);

  auto adjust = [&](float x, int e) {
    const unsigned w = count[e];
    const unsigned c = w & (kBias - 1u);
    if (c > 0u || (w & kPrompt)) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    if (c > 0u) x = __fsub_rn(__fsub_rn(x, __fmul_rn((float)c, freq)), pres);
    if (w & kBias) {
      for (int i = 0; i < s_bias_n; ++i)
        if (s_bias_id[i] == e) x = __fadd_rn(x, s_bias_v[i]);
    }
    return x;
  };

  for (int j = j0; j < j1; ++j) {
    const int64_t row = (int64_t)seq * a.rows + j;
    const T *in = static_cast<const T *>(a.logits) + row * a.logits_stride;
    O *out = static_cast<O *>(a.out) + row * a.out_stride;
    const unsigned *mask = a.mask ? reinterpret_cast<const unsigned *>(a.mask) + seq * a.mask_seq + j * a.mask_row
                                  : nullptr;
    // groups of eight from the 16-byte boundary at or before the slice's first element
    const int shift = (int)((reinterpret_cast<uintptr_t>(in + lo) & (8 * sizeof(T) - 1)) / sizeof(T));
    const bool out8 = ((reinterpret_cast<uintptr_t>(out + lo - shift)) & 15u) == 0;
    float x[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v0 = lo - shift + 8 * (k * kThreads + (int)threadIdx.x);
      if (v0 >= lo && v0 + 8 <= hi) {
        load8(in + v0, x[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = v0 + i >= lo && v0 + i < hi ? load1(in + v0 + i) : -INFINITY;
      }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v0 = lo - shift + 8 * (k * kThreads + (int)threadIdx.x);
      if (v0 >= hi) continue;
      if (counted) {
        const unsigned t = bits8(v0 - lo, a.slice / 32, [&](int w) { return touched[w]; });
        if (t) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (t >> i & 1) x[k][i] = adjust(x[k][i], v0 - lo + i);
        }
      }
      if (mask != nullptr) {
        const unsigned on = bits8(v0, (a.vocab + 31) / 32, [&](int w) { return __ldg(mask + w); });
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = on >> i & 1 ? x[k][i] : -INFINITY;
      }
    }
    if constexpr (PROBS) {
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // NaN counts as -inf, +inf as the largest finite number
          x[k][i] = fminf(fmaxf(x[k][i], -INFINITY), FLT_MAX);
          m = fmaxf(m, x[k][i]);
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float second = 0.f;  // the warp's sum, or the place of its first largest entry
      if (greedy) {
        int at = INT_MAX;
#pragma unroll
        for (int k = VPT - 1; k >= 0; --k)
#pragma unroll
          for (int i = 7; i >= 0; --i)
            if (x[k][i] == m) at = lo - shift + 8 * (k * kThreads + (int)threadIdx.x) + i;
        if (m == -INFINITY) at = INT_MAX;
        second = __int_as_float(__reduce_min_sync(0xffffffffu, at));
      } else {
        const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[k][i] = ex2_flush((x[k][i] - mm) * fac);
            second += x[k][i];
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) second += __shfl_xor_sync(0xffffffffu, second, o);
      }
      // every warp's pair to every thread block of the cluster; rows take turns with two
      // buffers, so a pair is read before the row after next overwrites it
      float2 *stat = s_stat[j & 1];
      if (lane < csize) dsmem_st_f32x2(dsmem_map(smem_u32(stat + crank * kWarps + warp), lane), m, second);
      sync_cluster();
      float M = -INFINITY;
      for (int i = lane; i < csize * kWarps; i += 32) M = fmaxf(M, stat[i].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      float mul = 0.f;
      int best = INT_MAX;
      if (greedy) {
        for (int i = lane; i < csize * kWarps; i += 32)
          if (stat[i].x == M) best = min(best, __float_as_int(stat[i].y));
        best = __reduce_min_sync(0xffffffffu, best);
      } else if (M != -INFINITY) {
        float sum = 0.f;
        for (int i = lane; i < csize * kWarps; i += 32) sum += stat[i].y * ex2_flush((stat[i].x - M) * fac);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        mul = m == -INFINITY ? 0.f : ex2_flush((m - M) * fac) / sum;
      }
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v0 = lo - shift + 8 * (k * kThreads + (int)threadIdx.x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = greedy ? (v0 + i == best ? 1.f : 0.f) : x[k][i] * mul;
      }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v0 = lo - shift + 8 * (k * kThreads + (int)threadIdx.x);
      if (out8 && v0 >= lo && v0 + 8 <= hi) {
        store8(out + v0, x[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (v0 + i >= lo && v0 + i < hi) store1(out + v0 + i, x[k][i]);
      }
    }
    if (a.drafts != nullptr && j + 1 < j1) {
      if (!PROBS) __syncthreads();  // (else the cluster barrier: every count of this row is read)
      if (threadIdx.x == 0) {
        const int v = __ldg(a.drafts + (int64_t)seq * (a.rows - 1) + j);
        if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
        if (v >= lo && v < hi) {
          count[v - lo] += 1u;
          touch(v - lo);
        }
      }
      __syncthreads();
    }
  }
  if (PROBS) sync_cluster();  // peers' shared memory stays until every pair has arrived
}

template <typename T, int VPT, bool PROBS>
cudaError_t launch_one(const LogitArgs &a, int cluster, cudaStream_t st) {
  auto kern = adjust_logits_kernel<T, VPT, PROBS>;
  const size_t smem = ((size_t)a.slice + a.slice / 32) * 4;
  static std::atomic<unsigned long long> opted{0};  // bit per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(opted.load(std::memory_order_acquire) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (VPT * kThreads * 8 + 32) / 32 * 33 * 4);
    if (e != cudaSuccess) return e;
    opted.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_seqs * a.row_groups * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, bool PROBS>
cudaError_t launch_slices(LogitArgs a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // slices of at most 16384 entries (two thread blocks an SM); smaller ones, and rows apart,
  // while the clusters do not fill the GPU twice
  int cluster = 1;
  while (cluster < kMaxCluster && (a.vocab > 16384 * cluster ||
                                   (a.vocab > 2048 * cluster && (int64_t)a.num_seqs * cluster < 2 * sms)))
    cluster *= 2;
  const int64_t units = (int64_t)a.num_seqs * cluster;
  a.row_groups = (int)std::min<int64_t>(a.rows, std::max<int64_t>(1, (2 * sms + units - 1) / units));
  a.slice = ((a.vocab + cluster - 1) / cluster + 31) / 32 * 32;
  if ((int64_t)units * a.row_groups >= (int64_t)1 << 31) return cudaErrorInvalidConfiguration;
  const int groups = (a.slice + 7) / 8 + 1;  // of eight elements, with a ragged one
  const int vpt = (groups + kThreads - 1) / kThreads;
  if (vpt <= 1) return launch_one<T, 1, PROBS>(a, cluster, st);
  if (vpt <= 3) return launch_one<T, 3, PROBS>(a, cluster, st);
  if (vpt <= 5) return launch_one<T, 5, PROBS>(a, cluster, st);
  return launch_one<T, 9, PROBS>(a, cluster, st);
}

}  // namespace
}  // namespace pa

extern "C" PA_API pa_status pa_adjust_logits(
    void *out, const void *logits, const int32_t *history, const int32_t *history_lens, const int32_t *prompt_lens,
    const int32_t *drafts, const float *repetition, const float *presence, const float *frequency,
    const int32_t *bias_ids, const float *bias_values, const int32_t *mask, const float *temperature, int num_seqs,
    int rows, int vocab, int max_history, int num_bias, pa_dtype dtype, int probs, int64_t out_stride,
    int64_t logits_stride, int64_t mask_seq_stride, int64_t mask_row_stride, void *stream) {
  using namespace pa;
  if (!out || !logits) return PA_ERR_INVALID_ARG;
  if ((history == nullptr) != (history_lens == nullptr) || (prompt_lens && !history)) return PA_ERR_INVALID_ARG;
  if ((bias_ids == nullptr) != (bias_values == nullptr) || (num_bias > 0 && !bias_ids)) return PA_ERR_INVALID_ARG;
  if (num_seqs < 0 || rows <= 0 || vocab <= 0 || max_history < 0 || num_bias < 0) return PA_ERR_INVALID_ARG;
  if (drafts && rows == 1) drafts = nullptr;  // no row stands behind a draft
  for (const void *p : {static_cast<const void *>(history), static_cast<const void *>(history_lens),
                        static_cast<const void *>(prompt_lens), static_cast<const void *>(drafts),
                        static_cast<const void *>(repetition), static_cast<const void *>(presence),
                        static_cast<const void *>(frequency), static_cast<const void *>(bias_ids),
                        static_cast<const void *>(bias_values), static_cast<const void *>(mask),
                        static_cast<const void *>(temperature)})
    if (!aligned4(p)) return PA_ERR_INVALID_ARG;
  if (dtype != PA_FP16 && dtype != PA_BF16 && dtype != PA_FP32) return PA_ERR_UNSUPPORTED;
  if (vocab > kMaxVocab || num_bias > kMaxBias) return PA_ERR_UNSUPPORTED;
  const int in_bytes = dtype == PA_FP32 ? 4 : 2, out_bytes = probs ? 4 : in_bytes;
  if (reinterpret_cast<uintptr_t>(logits) % in_bytes || reinterpret_cast<uintptr_t>(out) % out_bytes)
    return PA_ERR_INVALID_ARG;
  const int64_t total = (int64_t)num_seqs * rows;
  if (total >= (int64_t)1 << 27 || out_stride < vocab || logits_stride < vocab || out_stride >= (int64_t)1 << 40 ||
      logits_stride >= (int64_t)1 << 40)
    return PA_ERR_INVALID_ARG;
  if (mask && (mask_seq_stride < 0 || mask_row_stride < 0)) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  // in place, or apart
  const size_t out_n = ((total - 1) * out_stride + vocab) * out_bytes;
  const size_t in_n = ((total - 1) * logits_stride + vocab) * in_bytes;
  if (overlap(out, out_n, logits, in_n) && !(out == logits && out_bytes == in_bytes && out_stride == logits_stride))
    return PA_ERR_INVALID_ARG;
  const size_t words = ((size_t)vocab + 31) / 32, per = (size_t)num_seqs * 4;
  struct {
    const void *p;
    size_t n;
  } buf[] = {{history, per * max_history},
             {history_lens, per},
             {prompt_lens, per},
             {drafts, per * (rows - 1)},
             {repetition, per},
             {presence, per},
             {frequency, per},
             {bias_ids, per * num_bias},
             {bias_values, per * num_bias},
             {temperature, per},
             {mask, 4 * ((num_seqs - 1) * (size_t)mask_seq_stride + (rows - 1) * (size_t)mask_row_stride + words)}};
  for (const auto &b : buf)
    if (b.p && overlap(out, out_n, b.p, b.n)) return PA_ERR_INVALID_ARG;
  LogitArgs a;
  a.out = out;
  a.logits = logits;
  a.history = max_history > 0 ? history : nullptr;
  a.history_lens = history_lens;
  a.prompt_lens = prompt_lens;
  a.drafts = drafts;
  a.bias_ids = bias_ids;
  a.mask = mask;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_values = bias_values;
  a.temperature = temperature;
  a.num_seqs = num_seqs;
  a.rows = rows;
  a.vocab = vocab;
  a.max_history = max_history;
  a.num_bias = num_bias;
  a.slice = a.row_groups = 0;
  a.out_stride = out_stride;
  a.logits_stride = logits_stride;
  a.mask_seq = mask_seq_stride;
  a.mask_row = mask_row_stride;
  a.err = error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == PA_FP32)
    e = probs ? launch_slices<float, true>(a, st) : launch_slices<float, false>(a, st);
  else if (dtype == PA_FP16)
    e = probs ? launch_slices<__half, true>(a, st) : launch_slices<__half, false>(a, st);
  else
    e = probs ? launch_slices<__nv_bfloat16, true>(a, st) : launch_slices<__nv_bfloat16, false>(a, st);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
