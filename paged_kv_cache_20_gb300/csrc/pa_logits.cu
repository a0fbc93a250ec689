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
// A cluster of up to 16 thread blocks takes the rows of a sequence, each a slice of the
// vocabulary.  The softmax needs a row's maximum and sum over all slices, and exchanging them
// row by row left the GPU waiting.  So a thread block first reads up to kBatch rows and sums
// them, the cluster exchanges the sums of them all at once, and the rows are taken again, last
// ones first: the last are in shared memory still, the others are read again, in part from
// L2 (keeping them there by a cache hint: no faster).  Bulk copies bring the rows.  64 x 8
// rows of 131,071 bf16 logits take 145 us, where the bytes read and written once take 61: the
// schedulers issue in 59 % of the clocks, 344 warp instructions for 32 x 8 elements, and 34 clusters
// of 8 run at once, so that these are two rounds.  Against 174 us (before fp32 was stored in
// whole sectors, 26 us, and the list's inputs loaded at once): an exchange a row 183, batches of
// 4 rows 181, of 2 196, of 4 and 8 by turns 181; 256 threads 185, three thread blocks of them an
// SM 207; one thread block of 1024 threads an SM and two rows in registers 289; one barrier a
// row, with the bits of two rows side by side, 178 against 171 (registers).
// The entries that anything was counted for are few and lie anywhere: a slice keeps a list of
// them in ascending order with their counts, and one bit an entry.  The dense pass masks
// them out with the grammar's bits; the list's entries are gathered, adjusted and summed
// apart, a few a thread, and written over the dense pass's zeros.  The list serves all rows
// of a sequence: each draft joins it before the row behind it, and leaves it again on the
// way back.  (With every element testing its own bit and adjusting in place: 462 us.)
// A row of an odd vocabulary starts anywhere: a thread's eight elements are aligned to 16
// bytes of the row, not to the slice, whose ragged ends are masked.  Where the output's row does not
// start at the same element of 16 bytes, it is stored element by element: padded rows to dense
// ones of 131,071 take 311 us so, padded to padded 143.
// Above 131,072 entries 16 thread blocks a row: 64 x 8 of 151,936 take 238 us (floor 70), of
// 262,144 297 (121).
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
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

// The two halves of a cluster barrier that orders nothing: every thread block has started.
__device__ __forceinline__ void cluster_started() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_all_started() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;    // 8 up to kMostSlice * 8 entries; 16 is an opt-in
constexpr int kMostSlice = 16384;  // entries of a thread block
constexpr int kMaxStages = 2;
constexpr int kBatch = 8;  // rows that are summed before the exchange
constexpr int kMaxBias = 1024;
constexpr int kMaxVocab = kMostSlice * kMaxCluster;
constexpr int kMostShared = 226 * 1024;  // dynamic, beside less than 1 KiB of static
constexpr unsigned kPrompt = 1u << 31, kBias = 1u << 30;  // flags above an entry's count

// How a slice's shared memory is used (Room, below).
struct Modes {
  int wide, shared, stages;
};

struct LogitArgs {
  void *out;
  const void *logits;
  uint64_t logits_end;  // address past the last element
  const int32_t *history, *history_lens, *prompt_lens, *drafts, *bias_ids, *mask;
  const float *repetition, *presence, *frequency, *bias_values, *temperature;
  int num_seqs, rows, vocab, max_history, num_bias;
  int slice;      // entries of a thread block, a multiple of 32
  int listed;     // room for a slice's counted entries
  Modes modes;    // wide: their counts may pass 14 bits
  int row_groups;  // row groups of a sequence, each of its own cluster
  int64_t out_stride, logits_stride, mask_seq, mask_row;
  unsigned *err;
};

// Bits 0-3 and 4-7 of `on` as the top bits of four bytes each (the shifted copies of four
// bits do not meet); a byte permute then makes each a mask.
__device__ __forceinline__ uint32_t top_bits(unsigned four) { return four * 0x10204080u; }
// Bytes whose top bits they are: bytes 0, 0, 1, 1 (low pair) or 2, 2, 3, 3, each all its top bit.
__device__ __forceinline__ uint32_t pair_mask(uint32_t top, bool high) {
  uint32_t d;
  if (high)
    asm("prmt.b32 %0, %1, %1, 0xbbaa;" : "=r"(d) : "r"(top));
  else
    asm("prmt.b32 %0, %1, %1, 0x9988;" : "=r"(d) : "r"(top));
  return d;
}

// Eight elements of a row as they are read.
template <typename T>
struct Eight {  // fp16, bf16: pairs
  uint32_t w[4];
  static constexpr uint32_t kNegInf = Elt<T>::kMantBits == 10 ? 0xfc00fc00u : 0xff80ff80u;
  __device__ __forceinline__ void load(uint32_t at) {
    const uint4 v = lds128(at);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  // -inf where bit i of `on` is clear
  __device__ __forceinline__ void keep(unsigned on) {
    const uint32_t a = top_bits(on & 15u), b = top_bits(on >> 4);
    const uint32_t m[4] = {pair_mask(a, false), pair_mask(a, true), pair_mask(b, false), pair_mask(b, true)};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (w[i] & m[i]) | (kNegInf & ~m[i]);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // (of a NaN, the other)
    uint32_t d;
    if constexpr (Elt<T>::kMantBits == 10)
      asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
      asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ void no_nan() {  // NaN to -inf
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = max2(w[i], kNegInf);
  }
  __device__ __forceinline__ float largest() const {
    const float2 f = Elt<T>::to_f2(max2(max2(w[0], w[1]), max2(w[2], w[3])));
    return fmaxf(f.x, f.y);
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
  __device__ __forceinline__ void load(uint32_t at) {
    const uint4 a = lds128(at), b = lds128(at + 16);
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
  }
  __device__ __forceinline__ void keep(unsigned on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = on >> i & 1 ? v[i] : -INFINITY;
  }
  __device__ __forceinline__ void no_nan() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaxf(v[i], -INFINITY);
  }
  __device__ __forceinline__ float largest() const {
    return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
  }
};

// Four, with what writing them to fp32 takes.
template <typename T>
struct Four {
  uint32_t w[2];
  __device__ __forceinline__ void load(uint32_t at) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  }
  __device__ __forceinline__ void keep(unsigned on) {
    constexpr uint32_t inf = Eight<T>::kNegInf;
    const uint32_t a = top_bits(on & 15u), m0 = pair_mask(a, false), m1 = pair_mask(a, true);
    w[0] = (w[0] & m0) | (inf & ~m0);
    w[1] = (w[1] & m1) | (inf & ~m1);
  }
  __device__ __forceinline__ void no_nan() {
    w[0] = Eight<T>::max2(w[0], Eight<T>::kNegInf);
    w[1] = Eight<T>::max2(w[1], Eight<T>::kNegInf);
  }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    const float2 f = Elt<T>::to_f2(w[0]), g = Elt<T>::to_f2(w[1]);
    x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
  }
};
template <>
struct Four<float> {
  float v[4];
  __device__ __forceinline__ void load(uint32_t at) {
    const uint4 a = lds128(at);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
  }
  __device__ __forceinline__ void keep(unsigned on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = on >> i & 1 ? v[i] : -INFINITY;
  }
  __device__ __forceinline__ void no_nan() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaxf(v[i], -INFINITY);
  }
  __device__ __forceinline__ void get(float (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[i];
  }
};

template <typename T>
__device__ __forceinline__ float load1(const T *p) {
  if constexpr (sizeof(T) == 4)
    return *p;
  else
    return Elt<T>::to_f2(*reinterpret_cast<const uint16_t *>(p)).x;  // (the pair's upper half zero)
}
template <typename T>
__device__ __forceinline__ void store1(T *p, float x) {
  if constexpr (sizeof(T) == 4)
    *p = x;
  else
    *reinterpret_cast<uint16_t *>(p) = Elt<T>::from_f(x);
}
// Eight values to a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
  static_assert(sizeof(T) == 2, "fp32 is written in fours");
  __stcs(reinterpret_cast<uint4 *>(p), make_uint4(Elt<T>::from_f2(x[0], x[1]), Elt<T>::from_f2(x[2], x[3]),
                                                  Elt<T>::from_f2(x[4], x[5]), Elt<T>::from_f2(x[6], x[7])));
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

// Shared memory of a slice: rows' logits, a stage each; the counts that the list is made from
// (16 bits an entry, 32 where a history is too long for them), in the logits' place where
// that leaves room for another thread block (shared); a batch's statistics by warp, and by thread
// block; bits of counted entries, and of a row's mask and its dense elements, these with
// zeros before and behind (a warp's last group may start 248 elements past the slice); counts
// and places of the listed entries; biases (id, value).
constexpr int kOnBehind = 9;  // words
struct Room {
  int stage, step, counts, warps, blocks, touched, mask, on, cnt, bias_v, bias_id, list, total;
};
__host__ __device__ inline Room room_of(int slice, int listed, int num_bias, int cluster, int elt, Modes m) {
  const int counts = listed > 0 ? slice * (m.wide ? 4 : 2) : 0;
  const int stage = (slice * elt + 64 + 15) / 16 * 16;  // (whole groups around the slice's ragged ends)
  Room r;
  int at = 0;
  auto take = [&](int bytes) {
    const int was = at;
    at += (bytes + 15) / 16 * 16;
    return was;
  };
  r.step = stage;
  r.stage = r.counts = take(m.shared && counts > m.stages * stage ? counts : m.stages * stage);
  if (!m.shared)
    r.counts = take(counts);
  else if (m.stages > 1 && counts <= stage)
    r.counts += stage;  // the second row's: the first is on its way while the list is made
  r.warps = take(kBatch * kWarps * 8);
  r.blocks = take(kBatch * cluster * 8);
  r.touched = take(slice / 8);
  r.mask = take(slice / 8);
  r.on = take(slice / 8 + 4 + kOnBehind * 4);
  r.cnt = take(listed * 4);
  r.bias_v = take(num_bias * 4);
  r.bias_id = take(num_bias * 4);
  r.list = take(listed * 2);
  // a warp that any of its groups concerns reads them all: up to 255 elements and a shift of 7
  // past the slice, in the last stage past its end
  const int read = (m.stages - 1) * stage + (slice + 262) * elt;
  r.total = at > read ? at : (read + 15) / 16 * 16;
  return r;
}
constexpr int kNarrowMost = (1 << 14) - 1;  // counts of 16 bits: 14 and two flags

// VPT: groups of eight elements a thread holds.
template <typename T, int VPT, bool PROBS>
__global__ void __launch_bounds__(kThreads, 2) adjust_logits_kernel(const LogitArgs a) {
  using O = typename std::conditional<PROBS, float, T>::type;
  extern __shared__ __align__(16) uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_bar[kMaxStages];
  __shared__ int s_part[kWarps];
  __shared__ int s_bias_n;
  __shared__ float2 s_row[kBatch];  // of a batch's rows: the maximum, and the weights' factor or the one's place
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kMaxStages; ++i) mbar_init(smem_u32(&s_bar[i]), 1);
    fence_mbar_init();
    s_bias_n = 0;
  }
  if (PROBS) cluster_started();
  griddep_wait();
  griddep_launch_dependents();
  const int csize = (int)cluster_nctarank(), crank = (int)cluster_ctarank();
  const int unit = blockIdx.x / csize;
  const int seq = unit / a.row_groups, group = unit % a.row_groups;
  const int j0 = (int)((int64_t)a.rows * group / a.row_groups);
  const int j1 = (int)((int64_t)a.rows * (group + 1) / a.row_groups);
  const int lo = min(a.vocab, crank * a.slice), hi = min(a.vocab, lo + a.slice);
  const Room room = room_of(a.slice, a.listed, a.num_bias, csize, (int)sizeof(T), a.modes);
  const int stages = a.modes.stages;
  float2 *warp_stats = reinterpret_cast<float2 *>(s_raw + room.warps);    // [kBatch][kWarps]
  float2 *block_stats = reinterpret_cast<float2 *>(s_raw + room.blocks);  // [kBatch][cluster]
  unsigned *touched = reinterpret_cast<unsigned *>(s_raw + room.touched);
  unsigned *mask = reinterpret_cast<unsigned *>(s_raw + room.mask);
  unsigned *on = reinterpret_cast<unsigned *>(s_raw + room.on) + 1;
  unsigned *cnt = reinterpret_cast<unsigned *>(s_raw + room.cnt);
  float *bias_v = reinterpret_cast<float *>(s_raw + room.bias_v);
  int *bias_id = reinterpret_cast<int *>(s_raw + room.bias_id);
  uint16_t *list = reinterpret_cast<uint16_t *>(s_raw + room.list);
  const int words = a.slice / 32;  // at most kThreads: a word a thread
  const bool counted = a.listed > 0;

  // ---- a row's slice in shared memory: byte addr - base of the stage, base the boundary of
  // eight elements at or before the slice.  Copied in whole 16-byte pieces, also around
  // the slice's ends, but nothing outside the logits.
  constexpr uintptr_t kAlign = 8 * sizeof(T);
  const uintptr_t all0 = (reinterpret_cast<uintptr_t>(a.logits) + 15) & ~(uintptr_t)15;
  const uintptr_t all1 = (uintptr_t)a.logits_end & ~(uintptr_t)15;
  auto row_of = [&](int j) {
    return static_cast<const T *>(a.logits) + ((int64_t)seq * a.rows + j) * a.logits_stride;
  };
  auto copied = [&](const T *in, uintptr_t &c0, uintptr_t &c1) {
    c0 = reinterpret_cast<uintptr_t>(in + lo) & ~(uintptr_t)15;
    c1 = (reinterpret_cast<uintptr_t>(in + hi) + 15) & ~(uintptr_t)15;
    c0 = c0 > all0 ? c0 : all0;
    c1 = c1 < all1 ? c1 : all1;
    if (c1 < c0 || lo >= hi) c1 = c0;
  };
  auto fetch = [&](int j, int slot) {  // (one thread)
    const T *in = row_of(j);
    uintptr_t c0, c1;
    copied(in, c0, c1);
    const uintptr_t base = reinterpret_cast<uintptr_t>(in + lo) & ~(kAlign - 1);
    const uint32_t bar = smem_u32(&s_bar[slot]);
    mbar_arrive_expect_tx(bar, (uint32_t)(c1 - c0));
    if (c1 > c0)
      bulk_load(smem_u32(s_raw + room.stage + slot * room.step) + (uint32_t)(c0 - base),
                reinterpret_cast<const void *>(c0), (uint32_t)(c1 - c0), bar);
  };
  // the thread's word of a row's mask (entries past the vocabulary are not the slice's)
  const unsigned *mask_at = nullptr;
  if (a.mask != nullptr && lo + 32 * (int)threadIdx.x < hi)
    mask_at = reinterpret_cast<const unsigned *>(a.mask) + seq * a.mask_seq + (lo >> 5) + threadIdx.x;
  auto mask_word = [&](int j) { return mask_at != nullptr ? __ldg(mask_at + j * a.mask_row) : 0xffffffffu; };
  auto fetch_first = [&](int j) {  // (one thread) the first rows of those from j on
    for (int i = 0; i < min(j1 - j, stages); ++i) fetch(j + i, i);
  };
  // (of those that counts stand in the place of: all, or all but the first)
  const bool whole = a.modes.shared && room.counts == room.stage;
  auto fetch_rest = [&] {
    for (int i = whole ? 0 : 1; i < min(j1 - j0, stages); ++i) fetch(j0 + i, i);
  };
  if (threadIdx.x == 0) {
    if (!a.modes.shared)
      fetch_first(j0);
    else if (!whole)
      fetch(j0, 0);
  }
  // what the list and the rows take of the sequence is all on its way at once; of the history
  // also what may be past its length
  constexpr int kAhead = 8;
  int ids_ahead[kAhead], hist_n = 0, prompt = 0, bias_ahead = -1;
  float bias_v_ahead = 0.f;
  const int32_t *ids = a.history + (int64_t)seq * a.max_history;
  if (a.history != nullptr) {
    hist_n = __ldg(a.history_lens + seq);
    if (a.prompt_lens) prompt = __ldg(a.prompt_lens + seq);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = threadIdx.x + u * kThreads;
      ids_ahead[u] = i < a.max_history ? __ldg(ids + i) : -1;
    }
  }
  if (warp == 0 && lane < a.num_bias) {
    bias_ahead = __ldg(a.bias_ids + (int64_t)seq * a.num_bias + lane);
    bias_v_ahead = __ldg(a.bias_values + (int64_t)seq * a.num_bias + lane);
  }
  const float rep = a.repetition ? __ldg(a.repetition + seq) : 1.f;
  const float pres = a.presence ? __ldg(a.presence + seq) : 0.f;
  const float freq = a.frequency ? __ldg(a.frequency + seq) : 0.f;
  const float temp = a.temperature ? __ldg(a.temperature + seq) : 1.f;

  // ---- the list of counted entries
  int entries = 0;
  if (counted) {
    unsigned *dense = reinterpret_cast<unsigned *>(s_raw + room.counts);
    const bool wide = a.modes.wide != 0;
    for (int i = threadIdx.x; i < (wide ? a.slice : a.slice / 2); i += kThreads) dense[i] = 0u;
    if (threadIdx.x < words) touched[threadIdx.x] = 0u;
    __syncthreads();
    // an entry's count (in the low bits) or flag; narrow: two entries a word
    const unsigned prompt_bit = wide ? kPrompt : kPrompt >> 16, bias_bit = wide ? kBias : kBias >> 16;
    auto at_of = [&](int e) { return dense + (wide ? e : e >> 1); };
    auto up_of = [&](int e) { return wide ? 0 : (e & 1) * 16; };
    auto touch = [&](int e) { atomicOr(touched + (e >> 5), 1u << (e & 31)); };
    if (a.history != nullptr) {
      if ((hist_n < 0 || hist_n > a.max_history) && threadIdx.x == 0 && crank == 0) record_error(a.err, kErrCheck);
      const int n = min(max(hist_n, 0), a.max_history);
      auto put = [&](int i, int v) {
        if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
        if (v >= lo && v < hi) {
          const int e = v - lo;
          if (i < prompt)
            atomicOr(at_of(e), prompt_bit << up_of(e));
          else
            atomicAdd(at_of(e), 1u << up_of(e));
          touch(e);
        }
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if ((int)threadIdx.x + u * kThreads < n) put(threadIdx.x + u * kThreads, ids_ahead[u]);
#pragma unroll 4
      for (int i = threadIdx.x + kAhead * kThreads; i < n; i += kThreads) put(i, __ldg(ids + i));
    }
    if (a.drafts != nullptr)
      for (int i = threadIdx.x; i < j0; i += kThreads) {
        const int v = __ldg(a.drafts + (int64_t)seq * (a.rows - 1) + i);
        if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
        if (v >= lo && v < hi) {
          atomicAdd(at_of(v - lo), 1u << up_of(v - lo));
          touch(v - lo);
        }
      }
    // the slice's biases, in the list's order
    if (warp == 0 && a.num_bias > 0) {
      int n = 0;
      for (int i0 = 0; i0 < a.num_bias; i0 += 32) {
        const int i = i0 + lane;
        int v = bias_ahead;
        if (i0 > 0) v = i < a.num_bias ? __ldg(a.bias_ids + (int64_t)seq * a.num_bias + i) : -1;
        if (v >= a.vocab && crank == 0) record_error(a.err, kErrCheck);
        const bool mine = v >= lo && v < hi;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (mine) {
          const int at = n + __popc(who & ((1u << lane) - 1u));
          bias_id[at] = v - lo;
          bias_v[at] = i0 == 0 ? bias_v_ahead : __ldg(a.bias_values + (int64_t)seq * a.num_bias + i);
          atomicOr(at_of(v - lo), bias_bit << up_of(v - lo));
          touch(v - lo);
        }
        n += __popc(who);
      }
      if (lane == 0) s_bias_n = n;
    }
    __syncthreads();
    // ascending (its order is the order of the row's sums): a word a thread
    const unsigned mine = threadIdx.x < words ? touched[threadIdx.x] : 0u;
    int before = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += u;
    }
    if (lane == 31) s_part[warp] = before;
    before -= __popc(mine);
    __syncthreads();
    const int part = lane < kWarps ? s_part[lane] : 0;
    before += (int)__reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)part : 0u);
    entries = (int)__reduce_add_sync(0xffffffffu, (unsigned)part);
    for (unsigned b = mine; b; b &= b - 1u) {
      const int e = 32 * (int)threadIdx.x + __ffs(b) - 1;
      unsigned c = *at_of(e) >> up_of(e);
      if (!wide) c = (c & (bias_bit - 1u)) | (c & prompt_bit ? kPrompt : 0u) | (c & bias_bit ? kBias : 0u);
      list[before] = (uint16_t)e;
      cnt[before++] = c;
    }
    if (a.modes.shared) {  // the counts are read: their place may be copied to
      fence_proxy_async_smem();
      __syncthreads();
      if (threadIdx.x == 0) fetch_rest();
    }
  } else if (a.modes.shared && threadIdx.x == 0) {
    fetch_rest();
  }
  if (threadIdx.x <= kOnBehind) on[threadIdx.x == 0 ? -1 : words + (int)threadIdx.x - 1] = 0u;
  // which of the word's entries are the slice's
  const int ahead = hi - lo - 32 * (int)threadIdx.x;
  const unsigned valid = ahead >= 32 ? ~0u : ahead <= 0 ? 0u : (1u << ahead) - 1u;
  const bool greedy = PROBS && !(temp > 0.f);
  // the exponent's factor; kept finite and above zero (the least subnormal for an infinite
  // temperature), so that -inf stays -inf
  const float fac = fminf(fmaxf(1.4426950408889634f / temp, 1e-45f), FLT_MAX);
  __syncthreads();  // the copies' barriers and the list

  auto adjust = [&](float x, int e, unsigned w) {
    const unsigned c = w & (kBias - 1u);
    if (c > 0u || (w & kPrompt)) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    if (c > 0u) x = __fsub_rn(__fsub_rn(x, __fmul_rn((float)c, freq)), pres);
    if (w & kBias) {
      for (int i = 0; i < s_bias_n; ++i)
        if (bias_id[i] == e) x = __fadd_rn(x, bias_v[i]);
    }
    return x;
  };
  // 2^((x - m) fac) against a maximum m.  (One multiply-add with m fac rounded beforehand saves an
  // instruction an element and no time, and the largest weights, exact here, carry exp2's error
  // there: 5e-7 of a row against 1e-7.)
  auto near = [&](float x, float m) { return ex2_flush((x - m) * fac); };
  // The same of any m.  Above kFar x - m may overflow where logits of both signs lie near fp32's ends
  // (under temperatures as large that counts), half of it does not (a step that every element
  // would pay for: 64 x 8 rows of 131,071 146.0 us against 144.8); with an infinite m the entries
  // that reach it share the whole.
  constexpr float kFar = 1e30f;
  auto weight = [&](float x, float m) {
    if (m <= kFar) return near(x, m);
    if (m == INFINITY) return x == INFINITY ? 1.f : 0.f;
    const float half = fmaf(x, 0.5f, -0.5f * m) * fac;
    return ex2_flush(half + half);
  };

  // ---- the rows, one after the other in either direction
  constexpr int kStep = 8 * kThreads;
  unsigned phase = 0u;  // of each stage's next copy, a bit a stage
  const int32_t *drafts = a.drafts != nullptr ? a.drafts + (int64_t)seq * (a.rows - 1) : nullptr;
  auto draft_of = [&](int j) {  // the draft behind row j
    return drafts != nullptr && j >= j0 && j + 1 < j1 ? __ldg(drafts + j) : -1;
  };
  // A draft joins the list: `known` says that it is on it.  (Read by others behind the row's
  // barrier.)
  auto join = [&](int e, bool known) {
    if (known) {
      for (int i = threadIdx.x; i < entries; i += kThreads)
        if (list[i] == e) cnt[i] += 1u;
    } else {
      if (threadIdx.x == e >> 5) {
        touched[threadIdx.x] |= 1u << (e & 31);
        list[entries] = (uint16_t)e;
        cnt[entries] = 1u;
      }
      ++entries;
    }
  };
  // ... and leaves it: the last one that joined first.  One that brought its entry along left
  // it at the list's end with a count of one and no flag, which nothing else can have there.
  // (`last`, read before a barrier: it is such a one.)
  auto leave = [&](int e, bool last) {
    if (last) {
      if (threadIdx.x == e >> 5) touched[threadIdx.x] &= ~(1u << (e & 31));
      --entries;
    } else {
      for (int i = threadIdx.x; i < entries; i += kThreads)
        if (list[i] == e) cnt[i] -= 1u;
    }
  };
  const bool ragged = lo < hi && (reinterpret_cast<uintptr_t>(row_of(j0) + lo) < all0 ||
                                  reinterpret_cast<uintptr_t>(row_of(j1 - 1) + hi) > all1);
  struct Row {
    const uint8_t *stage;
    int shift, first;      // groups of eight start `shift` before the slice; the thread's group 0
    uint32_t base, up;     // its address, and its bits' place in the first word of
    const unsigned *bits;  // two that hold them
  };
  // The row at `in`, in stage `slot` (landed: it is there already), with mask word mw: to be worked on.
  auto begin = [&](const T *in, int slot, bool landed, unsigned mw) {
    Row r;
    uint8_t *stage = s_raw + room.stage + slot * room.step;
    r.stage = stage;
    r.shift = (int)((reinterpret_cast<uintptr_t>(in + lo) & (kAlign - 1)) / sizeof(T));
    r.first = lo - r.shift + 8 * (int)threadIdx.x;
    r.base = smem_u32(stage) + 8 * (uint32_t)sizeof(T) * threadIdx.x;
    r.up = 32u + (uint32_t)(r.first - lo);  // (from the word before `on`)
    r.bits = on + (int)(r.up >> 5) - 1;
    r.up &= 31u;
    if (threadIdx.x < words) {
      on[threadIdx.x] = valid & (counted ? mw & ~touched[threadIdx.x] : mw);
      mask[threadIdx.x] = mw;
    }
    // (one warp asks the copies' barrier: all of them asking take the scheduler's turns)
    if (!landed) {
      if (warp == 0 && !mbar_wait_bounded(smem_u32(&s_bar[slot]), phase >> slot & 1u)) record_error(a.err, kErrTimeout);
      phase ^= 1u << slot;
    }
    __syncthreads();
    // elements beside what was copied: the logits' own ragged ends
    if (ragged && !landed) {
      uintptr_t c0, c1;
      copied(in, c0, c1);
      const int e = threadIdx.x < 16 ? (int)threadIdx.x : hi - lo - 1 - ((int)threadIdx.x - 16);
      if (threadIdx.x < 32 && e >= 0 && e < hi - lo) {
        const uintptr_t g = reinterpret_cast<uintptr_t>(in + lo + e);
        if (g < c0 || g >= c1) reinterpret_cast<T *>(stage)[r.shift + e] = in[lo + e];
      }
      fence_proxy_async_smem();  // before the copy of another row
      __syncthreads();
    }
    return r;
  };
  // The thread's group k of a row, -inf for what is not dense or not the slice's; whether any
  // of the warp's groups k starts in the slice.
  auto dense = [&](const Row &r, int k) {
    Eight<T> x;
    x.load(r.base + k * (kStep * (uint32_t)sizeof(T)));
    x.keep(__funnelshift_r(r.bits[k * (kStep / 32)], r.bits[k * (kStep / 32) + 1], r.up) & 0xffu);
    if (PROBS) x.no_nan();
    return x;
  };
  const int warp_first = lo + 8 * 32 * __shfl_sync(0xffffffffu, warp, 0);
  auto there = [&](const Row &r, int k) { return warp_first + k * kStep < hi + r.shift; };
  // Entry i of the list, adjusted.
  auto adjusted = [&](const Row &r, int i) {
    const int e = list[i];
    float y = adjust(load1(reinterpret_cast<const T *>(r.stage) + r.shift + e), e, cnt[i]);
    if (a.mask != nullptr && !(mask[e >> 5] >> (e & 31) & 1u)) y = -INFINITY;
    return PROBS ? fmaxf(y, -INFINITY) : y;  // NaN counts as -inf
  };
  // The dense elements of a row, each group through `value`, to out (of the row): whole groups
  // with wide stores, if they lie on 16-byte boundaries there (fp32 in fours, so that a warp's
  // store fills whole 32-byte sectors; two stores of a thread's eight, half a sector each, took
  // 171 us for 64 x 8 rows of 131,071 where this takes 148); the slice's ragged ends, at
  // most seven elements each, by a thread each.  (With both in one loop a group's eight
  // single stores are predicated off one by one: 5 instructions an element.)
  auto write = [&](const Row &r, O *out, auto value) {
    O *o = out + r.first;
    if ((reinterpret_cast<uintptr_t>(out + lo - r.shift) & 15u) == 0) {
      if constexpr (sizeof(O) == 4) {
        const int in_warp = -4 * lane;  // its four from its eight: the warp's start and 4 lane
        const uint32_t at = r.base + in_warp * (int)sizeof(T);
        const uint32_t b = 32u + (uint32_t)(r.first + in_warp - lo);
        const unsigned *bits = on + (int)(b >> 5) - 1;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          if (!there(r, k)) continue;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int past = k * kStep + 128 * q, v0 = r.first + in_warp + past;
            Four<T> x;
            x.load(at + past * (uint32_t)sizeof(T));
            x.keep(__funnelshift_r(bits[past / 32], bits[past / 32 + 1], b));
            if (PROBS) x.no_nan();
            float f[4];
            x.get(f);
            value(v0, f);
            if (v0 >= lo && v0 + 4 <= hi) __stcs(reinterpret_cast<float4 *>(out + v0), make_float4(f[0], f[1], f[2], f[3]));
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          if (!there(r, k)) continue;
          const int v0 = r.first + k * kStep;
          float f[8];
          dense(r, k).get(f);
          value(v0, f);
          if (v0 >= lo && v0 + 8 <= hi) store8(o + k * kStep, f);
        }
      }
      // groups 0 and the last, unless they are whole
      const int n = hi - lo + r.shift;  // elements from group 0 on
      const bool head = r.shift > 0, tail = (n & 7) != 0 && (n > 8 || !head);
      if (threadIdx.x < 2 && (threadIdx.x == 0 ? head : tail)) {
        const int at = threadIdx.x == 0 ? 0 : n & ~7;  // elements from group 0 on
        Eight<T> x;
        x.load(smem_u32(r.stage) + at * (uint32_t)sizeof(T));
        const uint32_t b = 32u + (uint32_t)(at - r.shift);
        x.keep(__funnelshift_r(on[(int)(b >> 5) - 1], on[b >> 5], b) & 0xffu);
        if (PROBS) x.no_nan();
        const int v0 = lo - r.shift + at;
        float f[8];
        x.get(f);
        value(v0, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (v0 + i >= lo && v0 + i < hi) store1(out + v0 + i, f[i]);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < VPT; ++k) {
        if (!there(r, k)) continue;
        const int v0 = r.first + k * kStep;
        float f[8];
        dense(r, k).get(f);
        value(v0, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (v0 + i >= lo && v0 + i < hi) store1(o + k * kStep + i, f[i]);
      }
    }
  };
  // The stage of a row that was worked on: another row may come.
  auto release = [&](int slot, int next, bool more) {
    __syncthreads();
    if (threadIdx.x == 0 && more) fetch(next, slot);
  };

  if constexpr (!PROBS) {
    unsigned mw = mask_word(j0);
    int behind = draft_of(j0), slot = 0;
    const T *in = row_of(j0);
    O *out = static_cast<O *>(a.out) + ((int64_t)seq * a.rows + j0) * a.out_stride;
    for (int j = j0; j < j1; ++j, in += a.logits_stride, out += a.out_stride) {
      const Row r = begin(in, slot, false, mw);
      if (j + 1 < j1) mw = mask_word(j + 1);
      const int e = behind >= lo && behind < hi ? behind - lo : -1;
      if (behind >= a.vocab && crank == 0 && threadIdx.x == 0) record_error(a.err, kErrCheck);
      const bool known = e >= 0 && (touched[e >> 5] >> (e & 31) & 1u);
      behind = draft_of(j + 1);
      write(r, out, [](int, auto &) {});
      if (counted) {
        __syncthreads();  // the dense pass is written
        for (int i = threadIdx.x; i < entries; i += kThreads) store1(out + lo + list[i], adjusted(r, i));
      }
      release(slot, j + stages, j + stages < j1);
      if (e >= 0) join(e, known);
      if (++slot == stages) slot = 0;
    }
  } else {
    for (int b0 = j0; b0 < j1; b0 += kBatch) {
      const int b1 = min(j1, b0 + kBatch);
      // ---- forward: every warp's maximum of its part of a row, and the sum against it (or the
      // place of its first largest entry)
      if (b0 > j0) {
        if (threadIdx.x == 0)
          for (int i = 0; i < min(b1 - b0, stages); ++i) fetch(b0 + i, i);
      }
      unsigned mw = mask_word(b0);
      int behind = draft_of(b0), slot = 0;
      const T *in = row_of(b0);
      for (int j = b0; j < b1; ++j, in += a.logits_stride) {
        const Row r = begin(in, slot, false, mw);
        if (j + 1 < b1) mw = mask_word(j + 1);
        const int e = behind >= lo && behind < hi ? behind - lo : -1;
        if (behind >= a.vocab && crank == 0 && threadIdx.x == 0) record_error(a.err, kErrCheck);
        const bool known = e >= 0 && (touched[e >> 5] >> (e & 31) & 1u);
        behind = draft_of(j + 1);
        // (16-bit groups are kept for the second look, fp32 ones are taken again)
        constexpr bool kKeep = sizeof(T) == 2;
        Eight<T> x[kKeep ? VPT : 1];
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
          if (there(r, k)) {
            const Eight<T> g = dense(r, k);
            m = fmaxf(m, g.largest());
            if constexpr (kKeep) x[k] = g;
          }
        auto again = [&](int k, float (&f)[8]) {
          if constexpr (kKeep)
            x[k].get(f);
          else
            dense(r, k).get(f);
        };
        // the list's entries, as they come: their maximum, sum and place
        float ms = -INFINITY, ss = 0.f;
        int at = INT_MAX;
        for (int i = threadIdx.x; i < entries; i += kThreads) {
          const float y = adjusted(r, i);
          if (y == -INFINITY) continue;
          if (greedy) {
            const int v = lo + (int)list[i];
            if (y > ms || (y == ms && v < at)) at = v;
            ms = fmaxf(ms, y);
          } else if (y > ms) {
            ss = ss * weight(ms, y) + 1.f;
            ms = y;
          } else {
            ss += weight(y, ms);
          }
        }
        __syncwarp();
        m = fmaxf(m, ms);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float second = 0.f;
        if (greedy) {
          if (ms != m || m == -INFINITY) at = INT_MAX;
          if (m != -INFINITY) {
#pragma unroll
            for (int k = VPT - 1; k >= 0; --k) {
              if (!there(r, k)) continue;
              float f[8];
              again(k, f);
#pragma unroll
              for (int i = 7; i >= 0; --i)
                if (f[i] == m) at = min(at, r.first + k * kStep + i);
            }
          }
          __syncwarp();
          second = __int_as_float(__reduce_min_sync(0xffffffffu, at));
        } else {
          if (ms != -INFINITY) second = ss * weight(ms, m);
          if (m > kFar) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
              if (!there(r, k)) continue;
              float f[8];
              again(k, f);
#pragma unroll
              for (int i = 0; i < 8; ++i) second += weight(f[i], m);
            }
          } else if (m != -INFINITY) {
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
              if (!there(r, k)) continue;
              float f[8];
              again(k, f);
#pragma unroll
              for (int i = 0; i < 8; ++i) sum[i & 1] += near(f[i], m);
            }
            second += sum[0] + sum[1];
          }
          __syncwarp();
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) second += __shfl_xor_sync(0xffffffffu, second, o);
        }
        if (lane == 0) warp_stats[(j - b0) * kWarps + warp] = make_float2(m, second);
        release(slot, j + stages, j + stages < b1);
        if (e >= 0 && j + 1 < b1) join(e, known);
        if (++slot == stages) slot = 0;
      }
      // ---- the sums of all slices: warp r takes row r of the batch
      // of a warp's 32 pairs: the maximum, and the sum against it (or the least place of it)
      auto merged = [&](float2 v, float &M) {
        M = v.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (greedy)
          return __int_as_float(__reduce_min_sync(0xffffffffu, v.x == M ? __float_as_int(v.y) : INT_MAX));
        float sum = M == -INFINITY ? 0.f : v.y * weight(v.x, M);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        return sum;
      };
      const float2 none = make_float2(-INFINITY, greedy ? __int_as_float(INT_MAX) : 0.f);
      static_assert(kBatch <= kWarps && kWarps <= 32 && kMaxCluster <= 32, "a warp a row");
      if (b0 == j0) {
        cluster_all_started();
        __syncthreads();  // the warps' pairs
      } else {
        sync_cluster();  // ... and the peers have read the last batch's
      }
      const bool mine = warp < b1 - b0;
      if (mine) {
        float m;
        const float second = merged(lane < kWarps ? warp_stats[warp * kWarps + lane] : none, m);
        if (lane < csize) dsmem_st_f32x2(dsmem_map(smem_u32(block_stats + warp * csize + crank), lane), m, second);
      }
      sync_cluster();
      if (mine) {
        float m;
        const float second = merged(lane < csize ? block_stats[warp * csize + lane] : none, m);
        if (lane == 0)
          s_row[warp] = make_float2(m, !greedy ? 1.f / second : m == -INFINITY ? __int_as_float(INT_MAX) : second);
      }
      // ---- back: the last rows are in their stages still (s_row is read behind a row's barrier)
      mw = mask_word(b1 - 1);
      behind = draft_of(b1 - 2);
      float *out = static_cast<float *>(a.out) + ((int64_t)seq * a.rows + b1 - 1) * a.out_stride;
      for (int j = b1 - 1; j >= b0; --j, out -= a.out_stride) {
        in -= a.logits_stride;
        slot = slot == 0 ? stages - 1 : slot - 1;
        const Row r = begin(in, slot, j >= b1 - stages, mw);
        if (j > b0) mw = mask_word(j - 1);
        const int before = behind;  // the draft before this row, which leaves with it
        behind = draft_of(j - 2);
        const float2 stat = s_row[j - b0];
        const float M = stat.x, mul = stat.y;
        const int best = greedy ? __float_as_int(stat.y) : INT_MAX;
        if (!greedy && M <= kFar && M != -INFINITY) {
          write(r, out, [&](int, auto &f) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(f) / 4); ++i) f[i] = near(f[i], M) * mul;
          });
        } else {  // one, none, or those of a far maximum
          write(r, out, [&](int v0, auto &f) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(f) / 4); ++i)
              f[i] = greedy || M == -INFINITY ? (v0 + i == best ? 1.f : 0.f) : weight(f[i], M) * mul;
          });
        }
        if (counted) {
          __syncthreads();  // the dense pass is written
          for (int i = threadIdx.x; i < entries; i += kThreads) {
            const int e = list[i];
            float p;
            if (greedy || M == -INFINITY)
              p = lo + e == best ? 1.f : 0.f;
            else
              p = weight(adjusted(r, i), M) * mul;
            store1(out + lo + e, p);
          }
        }
        const int e = j > b0 && before >= lo && before < hi ? before - lo : -1;
        const bool last = e >= 0 && list[entries - 1] == e && cnt[entries - 1] == 1u;
        release(slot, j - stages, j - stages >= b0);
        if (e >= 0) leave(e, last);
      }
      // the next batch stands behind this one's drafts
      if (b1 < j1) {
        for (int j = b0; j < b1; ++j) {
          const int v = draft_of(j);
          if (v >= lo && v < hi) {
            const int e = v - lo;
            __syncthreads();
            const bool known = touched[e >> 5] >> (e & 31) & 1u;
            __syncthreads();
            join(e, known);
          }
        }
        __syncthreads();
      }
    }
  }
}

template <typename T, int VPT, bool PROBS>
cudaError_t launch_one(const LogitArgs &a, int cluster, cudaStream_t st) {
  auto kern = adjust_logits_kernel<T, VPT, PROBS>;
  static std::atomic<unsigned long long> opted{0};  // bit per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(opted.load(std::memory_order_acquire) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    opted.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_seqs * a.row_groups * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = room_of(a.slice, a.listed, a.num_bias, cluster, sizeof(T), a.modes).total;
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
  // slices of at most kMostSlice entries; smaller ones while the clusters do not fill the GPU
  // twice
  int cluster = 1;
  while (a.vocab > kMostSlice * cluster ||
         (cluster < 8 && a.vocab > 2048 * cluster && (int64_t)a.num_seqs * cluster < 2 * sms))
    cluster *= 2;
  a.slice = ((a.vocab + cluster - 1) / cluster + 31) / 32 * 32;
  // every entry of a slice may be counted, and no more than there are ids
  const int64_t ids = (int64_t)(a.history ? a.max_history : 0) + (a.drafts ? a.rows - 1 : 0) + a.num_bias;
  a.listed = (int)std::min<int64_t>(ids, a.slice);
  const int wide = ids > kNarrowMost;
  // Row groups: so many that the rounds of clusters take least, each of a group's rows and what a
  // thread block starts and ends with (as long as a row).  Places for clusters: nine tenths
  // of the SMs' (the GPU's parts hold whole ones: 34 of 8, two thread blocks an SM, were
  // counted).  A single round takes its time however few clusters are in it, since two share
  // their SMs all the same; of further rounds a part of the last one's gap (fitted to 1 to 128
  // sequences).  (As many groups as give every SM two thread blocks: 52 us for 16 x 8 rows of
  // 131,071, this 41; 32 and 25 for 8 x 8, 78 and 73 for 32 x 8, 111 and 96 for 40 x 8.)
  const bool two = room_of(a.slice, a.listed, a.num_bias, cluster, sizeof(T), Modes{wide, 1, 1}).total <= kMostShared / 2;
  const double places = std::max(1, sms * (two ? 18 : 9) / 10 / cluster);
  double least = 0.;
  for (int g = 1; g <= std::min(a.rows, 64); ++g) {
    const double w = (double)a.num_seqs * g / places, c = std::ceil(w);
    const double time = (c <= 1. ? 1. : w + (c - w) / (c * c - 1.)) * ((a.rows + g - 1) / g + 1);
    if (g == 1 || time < least) least = time, a.row_groups = g;
  }
  if ((int64_t)a.num_seqs * cluster * a.row_groups >= (int64_t)1 << 31) return cudaErrorInvalidConfiguration;
  const int per = (a.rows + a.row_groups - 1) / a.row_groups;
  // two thread blocks an SM where they fit, with a row ahead if that fits too
  const struct {
    Modes m;
    int most;
  } choice[] = {{{wide, 0, 2}, kMostShared / 2}, {{wide, 1, 2}, kMostShared / 2}, {{wide, 0, 1}, kMostShared / 2},
                {{wide, 1, 1}, kMostShared / 2}, {{wide, 0, 2}, kMostShared},     {{wide, 1, 2}, kMostShared},
                {{wide, 1, 1}, kMostShared}};
  for (const auto &c : choice) {
    if (c.m.stages > 1 && per == 1) continue;  // (a thread block has no second row)
    a.modes = c.m;
    if (room_of(a.slice, a.listed, a.num_bias, cluster, sizeof(T), c.m).total <= c.most) break;
  }
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
  a.logits_end = reinterpret_cast<uintptr_t>(logits) + in_n;
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
  a.modes = Modes{0, 0, 1};
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
