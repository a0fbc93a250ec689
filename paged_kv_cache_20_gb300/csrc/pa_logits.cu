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
// Bound by memory: a row is read once and written once.  A cluster of up to 16 thread blocks
// holds one row in registers, as it was read, each a slice of the vocabulary; a warp takes
// its part of the row against its own maximum, and one cluster barrier exchanges every
// warp's maximum and sum.
// The entries that anything was counted for are few and lie anywhere: a slice keeps their
// counts in shared memory, a list of them in ascending order, and one bit an entry.  The
// dense pass masks them out with the grammar's bits, two selects of registers an element;
// the list's entries are gathered, adjusted and summed apart, a few a thread, and written over
// the dense pass's zeros.  (With every element testing its own bit and adjusting in place,
// 64 x 8 rows of 131,071 took 462 us: the slice of the common tokens kept its whole cluster
// waiting.)  The list serves all rows of a sequence, each draft joining it before the next.
// A row of an odd vocabulary starts anywhere: a thread's eight elements are aligned to 16
// bytes of the row, not to the slice, whose ragged ends go by single elements.
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
constexpr int kMaxCluster = 16;    // 8 up to kMostSlice * 8 entries; 16 is an opt-in
constexpr int kMostSlice = 16384;  // entries of a thread block
constexpr int kMaxBias = 1024;
constexpr int kMaxVocab = kMostSlice * kMaxCluster;
constexpr unsigned kPrompt = 1u << 31, kBias = 1u << 30;  // flags above an entry's count

struct LogitArgs {
  void *out;
  const void *logits;
  const int32_t *history, *history_lens, *prompt_lens, *drafts, *bias_ids, *mask;
  const float *repetition, *presence, *frequency, *bias_values, *temperature;
  int num_seqs, rows, vocab, max_history, num_bias;
  int slice;      // entries of a thread block, a multiple of 32
  int listed;     // room for a slice's counted entries
  int row_groups;  // row groups of a sequence, each of its own cluster
  int64_t out_stride, logits_stride, mask_seq, mask_row;
  unsigned *err;
};

// Eight elements of a row as they are read.
template <typename T>
struct Eight {  // fp16, bf16: pairs
  uint32_t w[4];
  static constexpr uint32_t kNegInf = Elt<T>::kMantBits == 10 ? 0xfc00u : 0xff80u;
  __device__ __forceinline__ void load(const T *p) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  // elements i with bit i of `in` alone, -inf for the others
  __device__ __forceinline__ void load_some(const T *p, unsigned in) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = in >> i & 1 ? reinterpret_cast<const uint16_t *>(p)[i] : kNegInf;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | h[2 * i + 1] << 16;
  }
  // -inf where bit i of `on` is clear
  __device__ __forceinline__ void keep(unsigned on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = (on >> (2 * i) & 1 ? 0xffffu : 0u) | (on >> (2 * i + 1) & 1 ? 0xffff0000u : 0u);
      w[i] = (w[i] & m) | ((kNegInf | kNegInf << 16) & ~m);
    }
  }
  __device__ __forceinline__ void no_nan() {  // NaN to -inf (the other operand is taken)
    const uint32_t neg = kNegInf | kNegInf << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (Elt<T>::kMantBits == 10)
        asm("max.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(neg));
      else
        asm("max.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(neg));
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elt<T>::to_f2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void load(const float *p) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void load_some(const float *p, unsigned in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = in >> i & 1 ? p[i] : -INFINITY;
  }
  __device__ __forceinline__ void keep(unsigned on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = on >> i & 1 ? v[i] : -INFINITY;
  }
  __device__ __forceinline__ void no_nan() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaxf(v[i], -INFINITY);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
  }
};

template <typename T>
__device__ __forceinline__ float load1(const T *p) {
  if constexpr (sizeof(T) == 4)
    return *p;
  else
    return Elt<T>::to_f2(*reinterpret_cast<const uint16_t *>(p)).x;
}
template <typename T>
__device__ __forceinline__ void store1(T *p, float x) {
  if constexpr (sizeof(T) == 4)
    *p = x;
  else
    *reinterpret_cast<uint16_t *>(p) = Elt<T>::from_f(x);
}
// Eight values: whole groups at 16-byte boundaries, else the elements of `in`.
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8], bool whole, unsigned in) {
  if (whole) {
    if constexpr (sizeof(T) == 4) {
      __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
      __stcs(reinterpret_cast<uint4 *>(p), make_uint4(Elt<T>::from_f2(x[0], x[1]), Elt<T>::from_f2(x[2], x[3]),
                                                      Elt<T>::from_f2(x[4], x[5]), Elt<T>::from_f2(x[6], x[7])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in >> i & 1) store1(p + i, x[i]);
  }
}

// 2^x, subnormal results to zero (a probability below 2^-126 of the largest)
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

// Elements of the group at v0 that lie in [lo, hi), as bits.
__device__ __forceinline__ unsigned inside(int v0, int lo, int hi) {
  unsigned in = 0xffu;
  if (v0 < lo) in &= 0xffu << min(8, lo - v0);
  if (v0 + 8 > hi) in &= v0 < hi ? 0xffu >> (v0 + 8 - hi) : 0u;
  return in & 0xffu;
}

// Shared memory of a slice: counts [slice], bits [slice / 32], list [listed] (16 bits each),
// adjusted values [listed], biases (id, value) [num_bias].
__host__ __device__ __forceinline__ size_t slice_bytes(int slice, int listed, int num_bias) {
  return (size_t)slice * 4 + slice / 8 + (size_t)listed * 2 + (size_t)listed * 4 + (size_t)num_bias * 8;
}

// VPT: groups of eight elements a thread holds.
template <typename T, int VPT, bool PROBS>
__global__ void __launch_bounds__(kThreads, 2) adjust_logits_kernel(const LogitArgs a) {
  using O = typename std::conditional<PROBS, float, T>::type;
  extern __shared__ unsigned s_words[];
  __shared__ __align__(8) float2 s_stat[2][kMaxCluster * kWarps];
  __shared__ int s_part[kWarps];
  __shared__ int s_bias_n, s_listed;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int csize = (int)cluster_nctarank(), crank = (int)cluster_ctarank();
  const int unit = blockIdx.x / csize;
  const int seq = unit / a.row_groups, group = unit % a.row_groups;
  const int j0 = (int)((int64_t)a.rows * group / a.row_groups);
  const int j1 = (int)((int64_t)a.rows * (group + 1) / a.row_groups);
  const int lo = min(a.vocab, crank * a.slice), hi = min(a.vocab, lo + a.slice);
  unsigned *count = s_words, *touched = count + a.slice;
  float *adj = reinterpret_cast<float *>(touched + a.slice / 32);
  float *bias_v = adj + a.listed;
  int *bias_id = reinterpret_cast<int *>(bias_v + a.num_bias);
  uint16_t *list = reinterpret_cast<uint16_t *>(bias_id + a.num_bias);
  const bool counted = a.listed > 0;

  int entries = 0;  // on the list
  if (counted) {
    for (int i = threadIdx.x; i < a.slice + a.slice / 32; i += kThreads) s_words[i] = 0u;
    if (threadIdx.x == 0) s_bias_n = 0;
    __syncthreads();
    auto touch = [&](int e) { atomicOr(touched + (e >> 5), 1u << (e & 31)); };
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
    if (warp == 0 && a.num_bias > 0) {
      int n = 0;
      for (int i0 = 0; i0 < a.num_bias; i0 += 32) {
        const int i = i0 + lane;
        const int v = i < a.num_bias ? __ldg(a.bias_ids + (int64_t)seq * a.num_bias + i) : -1;
        if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
        const bool mine = v >= lo && v < hi;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (mine) {
          const int at = n + __popc(who & ((1u << lane) - 1u));
          bias_id[at] = v - lo;
          bias_v[at] = __ldg(a.bias_values + (int64_t)seq * a.num_bias + i);
          atomicOr(count + (v - lo), kBias);
          touch(v - lo);
        }
        n += __popc(who);
      }
      if (lane == 0) s_bias_n = n;
    }
    __syncthreads();
    // the list, ascending (its order is the order of the row's sums): each thread's words
    const int words = a.slice / 32, per = (words + kThreads - 1) / kThreads;
    const int w0 = min(words, (int)threadIdx.x * per), w1 = min(words, w0 + per);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(touched[w]);
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += u;
    }
    if (lane == 31) s_part[warp] = before;
    before -= mine;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_part[w];
      entries += s_part[w];
    }
    for (int w = w0; w < w1; ++w)
      for (unsigned b = touched[w]; b; b &= b - 1u) list[before++] = (uint16_t)(32 * w + __ffs(b) - 1);
    if (threadIdx.x == 0) s_listed = entries;
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
        if (bias_id[i] == e) x = __fadd_rn(x, bias_v[i]);
    }
    return x;
  };
  // 2^((x - m) fac) against a maximum m; with an infinite m the entries that reach it
  auto weight = [&](float x, float m) {
    return m == INFINITY ? (x == INFINITY ? 1.f : 0.f) : ex2_flush((x - m) * fac);
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
    const int first = lo - shift + 8 * (int)threadIdx.x;  // of the thread's group 0
    constexpr int kStep = 8 * kThreads;
    Eight<T> x[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v0 = first + k * kStep;
      if (v0 >= lo && v0 + 8 <= hi)
        x[k].load(in + v0);
      else
        x[k].load_some(in + v0, inside(v0, lo, hi));
    }
    // the list's entries
    float m = -INFINITY;
    for (int i = threadIdx.x; i < entries; i += kThreads) {
      const int e = list[i];
      float y = adjust(load1(in + lo + e), e);
      if (mask != nullptr && !(__ldg(mask + ((lo + e) >> 5)) >> ((lo + e) & 31) & 1)) y = -INFINITY;
      if (PROBS) y = fmaxf(y, -INFINITY);  // NaN counts as -inf
      adj[i] = y;
      m = fmaxf(m, y);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v0 = first + k * kStep;
      if (v0 < hi) {
        unsigned on = 0xffu;
        if (mask != nullptr) on = bits8(v0, (a.vocab + 31) / 32, [&](int w) { return __ldg(mask + w); });
        if (counted) on &= ~bits8(v0 - lo, a.slice / 32, [&](int w) { return touched[w]; });
        if (on != 0xffu) x[k].keep(on);
        if (PROBS) x[k].no_nan();
      }
    }
    float mul = 0.f, M = -INFINITY;
    int best = INT_MAX;
    if constexpr (PROBS) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float f[8];
        x[k].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, f[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float second = 0.f;  // the warp's sum, or the place of its first largest entry
      if (greedy) {
        int at = INT_MAX;
        if (m != -INFINITY) {
#pragma unroll
          for (int k = VPT - 1; k >= 0; --k) {
            float f[8];
            x[k].get(f);
#pragma unroll
            for (int i = 7; i >= 0; --i)
              if (f[i] == m) at = first + k * kStep + i;
          }
          for (int i = threadIdx.x; i < entries; i += kThreads)
            if (adj[i] == m) at = min(at, lo + (int)list[i]);
        }
        second = __int_as_float(__reduce_min_sync(0xffffffffu, at));
      } else if (m != -INFINITY) {
        for (int i = threadIdx.x; i < entries; i += kThreads) second += weight(adj[i], m);
        if (m == INFINITY) {
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            float f[8];
            x[k].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) second += f[i] == INFINITY ? 1.f : 0.f;
          }
        } else {
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            float f[8];
            x[k].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) second += ex2_flush((f[i] - m) * fac);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) second += __shfl_xor_sync(0xffffffffu, second, o);
      }
      // every warp's pair to every thread block of the cluster; rows take turns with two
      // buffers, so a pair is read before the row after next overwrites it
      float2 *stat = s_stat[j & 1];
      if (lane < csize) dsmem_st_f32x2(dsmem_map(smem_u32(stat + crank * kWarps + warp), lane), m, second);
      sync_cluster();
      for (int i = lane; i < csize * kWarps; i += 32) M = fmaxf(M, stat[i].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      if (greedy) {
        for (int i = lane; i < csize * kWarps; i += 32)
          if (stat[i].x == M) best = min(best, __float_as_int(stat[i].y));
        best = __reduce_min_sync(0xffffffffu, best);
      } else if (M != -INFINITY) {
        float sum = 0.f;
        for (int i = lane; i < csize * kWarps; i += 32) sum += stat[i].y * weight(stat[i].x, M);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        mul = 1.f / sum;
      }
    } else if (entries > 0) {
      __syncthreads();  // in place: the list's logits are read before the row is written
    }
    const bool none = PROBS && M == -INFINITY;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v0 = first + k * kStep;
      float f[8];
      x[k].get(f);
      if constexpr (PROBS) {
        if (greedy || none) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = v0 + i == best ? 1.f : 0.f;
        } else if (M == INFINITY) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = f[i] == INFINITY ? mul : 0.f;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = ex2_flush((f[i] - M) * fac) * mul;
        }
      }
      if (v0 < hi) {
        const unsigned part = inside(v0, lo, hi);
        store8(out + v0, f, out8 && part == 0xffu, part);
      }
    }
    if (entries > 0 || a.drafts != nullptr) {
      __syncthreads();  // the dense pass is written, and every bit and count of this row read
      for (int i = threadIdx.x; i < entries; i += kThreads) {
        const int v = lo + (int)list[i];
        float y = adj[i];
        if (PROBS) y = greedy || none ? (v == best ? 1.f : 0.f) : weight(y, M) * mul;
        store1(out + v, y);
      }
      if (a.drafts != nullptr && j + 1 < j1) {
        if (threadIdx.x == 0) {
          const int v = __ldg(a.drafts + (int64_t)seq * (a.rows - 1) + j);
          if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
          if (v >= lo && v < hi) {
            const int e = v - lo;
            count[e] += 1u;
            if (!(touched[e >> 5] >> (e & 31) & 1)) {
              touched[e >> 5] |= 1u << (e & 31);
              list[s_listed] = (uint16_t)e;
              s_listed += 1;
            }
          }
        }
        __syncthreads();
        entries = s_listed;
      }
    }
  }
  if (PROBS) sync_cluster();  // peers' shared memory stays until every pair has arrived
}

template <typename T, int VPT, bool PROBS>
cudaError_t launch_one(const LogitArgs &a, int cluster, cudaStream_t st) {
  auto kern = adjust_logits_kernel<T, VPT, PROBS>;
  constexpr int kMost = std::min(VPT * kThreads * 8, kMostSlice);  // entries of this kernel's slices
  static std::atomic<unsigned long long> opted{0};  // bit per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(opted.load(std::memory_order_acquire) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)slice_bytes(kMost, kMost, kMaxBias));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    opted.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_seqs * a.row_groups * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.listed > 0 ? slice_bytes(a.slice, a.listed, a.num_bias) : 0;
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
  // slices of at most kMostSlice entries (two thread blocks an SM); smaller ones, and rows apart,
  // while the clusters do not fill the GPU twice
  int cluster = 1;
  while (a.vocab > kMostSlice * cluster ||
         (cluster < 8 && a.vocab > 2048 * cluster && (int64_t)a.num_seqs * cluster < 2 * sms))
    cluster *= 2;
  const int64_t units = (int64_t)a.num_seqs * cluster;
  a.row_groups = (int)std::min<int64_t>(a.rows, std::max<int64_t>(1, (2 * sms + units - 1) / units));
  a.slice = ((a.vocab + cluster - 1) / cluster + 31) / 32 * 32;
  if ((int64_t)units * a.row_groups >= (int64_t)1 << 31) return cudaErrorInvalidConfiguration;
  // every entry of a slice may be counted, and no more than there are ids
  const int64_t ids = (int64_t)(a.history ? a.max_history : 0) + (a.drafts ? a.rows - 1 : 0) + a.num_bias;
  a.listed = (int)std::min<int64_t>(ids, a.slice);
  const int groups = (a.slice + 7) / 8 + 1;  // of eight elements, with a ragged one
  const int vpt = (groups + kThreads - 1) / kThreads;
  if (vpt <= 1) return launch_one<T, 1, PROBS>(a, cluster, st);
  if (vpt <= 3) return launch_one<T, 3, PROBS>(a, cluster, st);
  return launch_one<T, 5, PROBS>(a, cluster, st);
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
  a.slice = a.row_groups = a.listed = 0;
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
