// pa_rope.cu -- rotary positions of one or several axes, applied to q and to the new
// K rows on their way into the paged cache (V rows go along unrotated).
//
// Pair i of a head (0 <= i < rotary_dim / 2) holds elements (i, i + rotary_dim / 2),
// or (2i, 2i + 1) when interleaved, and turns by
//   theta = positions[axis_i][token] * f_i:
//   a' = a cos(theta) - b sin(theta),  b' = b cos(theta) + a sin(theta)
// in fp32, rounded once to the 16-bit type (or divided by the head's scale and
// rounded once to e4m3 for an FP8 cache).  Elements past rotary_dim are copied.
//
// The angle.  A position of 10^6 times a frequency near 1 needs 2^20 more than the
// 24 bits of fp32 to keep its fraction of a turn, and GB300's fp64 rate is far too low
// to spend on it.  So frequencies arrive as F_i = 2^64 f_i / (2 pi), an integer: the
// product position * F_i modulo 2^64 is the fraction of a turn, exact in integer
// arithmetic up to |position| * 2^-65 turns from F_i's own rounding.  Its upper 32
// bits, as a signed number of half turns in [-1, 1), go to sincospif.
//
// Bound by DRAM: every byte of q, k, v once in and once out.  A CTA walks tokens, each
// thread on the same items of every token.  A token's q, k and v rows come by three bulk
// copies into a ring of stages in shared memory, so that two tokens a CTA are in flight
// without registers (which lets three 384-thread CTAs share an SM; two measured 2 %
// slower, four spill); the next token's angles are worked out while the current one is
// rotated and stored, and one barrier per token hands them over and the stage back.
// 8192 tokens of 32/8 heads 33.8 us (6.0 TB/s), 4099 of 32/32 into an FP8 cache 31.7
// (5.3 TB/s); with loads to registers a token ahead 34.3 and 38.3; with one CTA per token
// 42.5 and 37.6.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "pa_decode.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace {

struct RopeArgs {
  uint16_t *q_out;
  const uint16_t *q, *k, *v;
  void *k_cache, *v_cache;
  const int32_t *positions;     // [num_axes][n_tokens]
  const int64_t *slot_mapping;  // [n_tokens]
  const int64_t *turns;         // [rotary_dim / 2], units of 2^-64 turns per position
  const int32_t *pair_axis;     // [rotary_dim / 2]
  int64_t q_out_stride, q_stride, k_stride, v_stride;  // elements between tokens
  int64_t num_slots;
  // heads of this launch (the pointers stand at its first ones); KV heads of a cache block
  int num_q_heads, num_kv_heads, cache_heads;
  int n_tokens, half, num_axes, block_shift, stages;
  const float *k_scale, *v_scale;
  unsigned *err;
};

// The angles of a token in shared memory, (cos, sin) a pair, placed so that the eight
// lanes of a 16-byte read phase, which hold consecutive chunks, fall on eight different
// bank groups (pair after pair they would share two or four): halves apart, pairs
// 8 c + 2 q and + 1 at [q][c]; adjacent, pairs 4 j + 2 q and + 1 at [q][j].
template <bool ADJ>
__device__ __forceinline__ int angle_at(int pair) {
  return ADJ ? 2 * (16 * ((pair >> 1) & 1) + (pair >> 2)) + (pair & 1)
             : 2 * (8 * ((pair >> 1) & 3) + (pair >> 3)) + (pair & 1);
}

// Eight rotated pairs, 8 c .. 8 c + 7: a (16 bytes of first elements) and b (of second
// elements); fp32 results in x (a') and y (b').
template <typename T>
__device__ __forceinline__ void rotate8(const uint4 a, const uint4 b, const float2 *cs, int c,
                                        float (&x)[8], float (&y)[8]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 fa = pa::Elt<T>::to_f2(wa[i]), fb = pa::Elt<T>::to_f2(wb[i]);
    const float4 t = *reinterpret_cast<const float4 *>(cs + 2 * (8 * i + c));  // of two pairs
    x[2 * i] = fmaf(fa.x, t.x, -fb.x * t.y);
    y[2 * i] = fmaf(fb.x, t.x, fa.x * t.y);
    x[2 * i + 1] = fmaf(fa.y, t.z, -fb.y * t.w);
    y[2 * i + 1] = fmaf(fb.y, t.z, fa.y * t.w);
  }
}

// Four adjacent pairs, chunk j of a head (elements 8 j .. 8 j + 7).
template <typename T>
__device__ __forceinline__ void rotate4_adjacent(const uint4 a, const float2 *cs, int j, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = pa::Elt<T>::to_f2(w[2 * i]), g = pa::Elt<T>::to_f2(w[2 * i + 1]);
    const float4 t = *reinterpret_cast<const float4 *>(cs + 2 * (16 * i + j));
    x[4 * i] = fmaf(f.x, t.x, -f.y * t.y);
    x[4 * i + 1] = fmaf(f.y, t.x, f.x * t.y);
    x[4 * i + 2] = fmaf(g.x, t.z, -g.y * t.w);
    x[4 * i + 3] = fmaf(g.y, t.z, g.x * t.w);
  }
}

template <typename T>
__device__ __forceinline__ void widen8(const uint4 a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = pa::Elt<T>::to_f2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  return make_uint4(pa::Elt<T>::from_f2(x[0], x[1]), pa::Elt<T>::from_f2(x[2], x[3]),
                    pa::Elt<T>::from_f2(x[4], x[5]), pa::Elt<T>::from_f2(x[6], x[7]));
}

// Eight e4m3 codes of x / scale.  With r = 1 / scale rounded, q = x r and the exact
// remainder q scale - x, q - remainder r is the correctly rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990)
// where nothing overflows or underflows: a positive scale within 2^+-60 and |x| up to
// 2^60 scale leave only quotients far below e4m3's smallest step to underflow, and those
// keep their sign.  Everything else is divided.  (Three operations a value against about
// twenty: the quantising of 33 M values bounded the kernel.)
struct Divisor {
  float scale, r, most;  // most: largest |x| of the short way
  __device__ __forceinline__ void set(float s) {
    scale = s;
    r = 1.f / s;
    most = s >= 0x1p-60f && s <= 0x1p60f ? s * 0x1p60f : -1.f;
  }
};

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], const Divisor &d) {
  // (NaN passes the test: it stays NaN either way)
  float m = fmaxf(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
  for (int i = 2; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  float y[8];
  if (m <= d.most) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x[i] * d.r;
      y[i] = fmaf(-fmaf(q, d.scale, -x[i]), d.r, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] / d.scale;
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = pa::f32x2_to_e4m3x2(y[2 * i], y[2 * i + 1]);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

constexpr int kMaxHalf = 64;  // rotary pairs per head at most (head_dim 128)
constexpr int kMaxAxes = 32;
constexpr int kThreads = 384;  // at most
constexpr int kPer = 2;        // items of a thread
constexpr int kMaxHeads = kThreads * kPer / 8;  // of a launch, at head_dim 128: 96
constexpr int kMaxStages = 2;  // (3 and 4 measured the same and 3 % slower)
constexpr int kStageMemory = 208 * 1024;  // of an SM's shared memory, for stages
constexpr int kResident = 1152;           // threads an SM holds (56 registers each)

// An item is two 16-byte chunks of one head.  The chunks that are rotated (and, apart from
// them, those that are copied: V, and elements past rotary_dim) are paired first half with
// second half, so that consecutive lanes read and write consecutive chunks, and with the
// halves apart a pair's two elements are in one item.  A token's items in order: rotated
// ones of q and of K, copied ones of q, K and V (so that a warp's lanes do the same).
// Thread i takes items u blockDim + i of tokens blockIdx.x,
// + gridDim.x, ...
template <typename T, int D, bool ADJ, bool KV8>
__global__ void __launch_bounds__(kThreads, 3) rope_append_kernel(const RopeArgs a) {
  constexpr int kItems = D / 16;  // items of a head
  extern __shared__ __align__(128) uint8_t s_stage[];
  __shared__ __align__(8) uint64_t s_full[kMaxStages];
  __shared__ __align__(16) float2 cs[2][kMaxHalf];
  __shared__ int64_t s_turn[kMaxHalf];
  __shared__ int s_axis[kMaxHalf], s_pos[2][kMaxAxes];
  __shared__ int64_t s_kv[3];  // the token's byte offset in the caches, -1: none
  __shared__ int s_failed;
  const int tid = threadIdx.x;
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int64_t G = gridDim.x;
  const uint32_t q_bytes = (uint32_t)hq * (D * 2), kv_bytes = (uint32_t)hkv * (D * 2);
  const uint32_t stage_bytes = q_bytes + 2 * kv_bytes;
  if (tid == 0) {
    s_failed = 0;
    for (int i = 0; i < a.stages; ++i) pa::mbar_init(pa::smem_u32(&s_full[i]), 1);
    pa::fence_mbar_init();
  }
  pa::griddep_wait();
  pa::griddep_launch_dependents();

  // token t into stage i (thread 0)
  auto fetch = [&](int64_t t, int i) {
    const uint32_t bar = pa::smem_u32(&s_full[i]);
    const uint32_t to = pa::smem_u32(s_stage) + i * stage_bytes;
    pa::mbar_arrive_expect_tx(bar, stage_bytes);
    if (q_bytes) pa::bulk_load(to, a.q + t * a.q_stride, q_bytes, bar);
    if (kv_bytes) {
      pa::bulk_load(to + q_bytes, a.k + t * a.k_stride, kv_bytes, bar);
      pa::bulk_load(to + q_bytes + kv_bytes, a.v + t * a.v_stride, kv_bytes, bar);
    }
  };
  int64_t t = blockIdx.x;
  if (tid == 0)
    for (int i = 0; i < a.stages; ++i)
      if (t + i * G < a.n_tokens) fetch(t + i * G, i);

  // this thread's items, the same of every token: where they lie in a stage and where they
  // go to (bytes, the token's own offset apart), kind 0 q, 1 K, 2 V, 3 none
  uint32_t src[kPer];
  char *dst[kPer];
  int kind[kPer], d0[kPer], d1[kPer], pairs[kPer];  // d0, d1: the chunks' elements; pairs: < 0 copied
  Divisor div[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    int it = u * blockDim.x + tid;
    const int rot_items = a.half / 8, copied = kItems - rot_items;
    const bool rot = it < (hq + hkv) * rot_items;
    int h = 0, c = 0, n = rot_items;  // item c of n of its kind in head h
    kind[u] = 3;
    if (rot) {
      h = it / rot_items, c = it % rot_items;
      kind[u] = h < hq ? 0 : 1;
    } else if ((it -= (hq + hkv) * rot_items) < (hq + hkv) * copied) {
      n = copied;
      h = it / copied, c = it % copied;
      kind[u] = h < hq ? 0 : 1;
    } else if ((it -= (hq + hkv) * copied) < hkv * kItems) {
      n = kItems;
      h = it / kItems, c = it % kItems;
      kind[u] = 2;
    }
    const int chunk = rot || kind[u] == 2 ? c : 2 * rot_items + c;
    d0[u] = 8 * chunk;
    d1[u] = 8 * (chunk + n);
    pairs[u] = rot ? c : -1;
    src[u] = pa::smem_u32(s_stage) + (kind[u] == 2 ? q_bytes + kv_bytes : 0u) + (uint32_t)h * (D * 2);
    if (kind[u] == 1) h -= hq;
    dst[u] = kind[u] == 0 ? reinterpret_cast<char *>(a.q_out + (int64_t)h * D)
                          : static_cast<char *>(kind[u] == 1 ? a.k_cache : a.v_cache) +
                                ((int64_t)h << a.block_shift) * (D * (KV8 ? 1 : 2));
    if (KV8) div[u].set(kind[u] == 1 ? __ldg(a.k_scale + h) : kind[u] == 2 ? __ldg(a.v_scale + h) : 1.f);
  }
  auto angles = [&](int buf) {
    for (int i = tid; i < a.half; i += blockDim.x) {
      const uint64_t turn = (uint64_t)(int64_t)s_pos[buf][s_axis[i]] * (uint64_t)s_turn[i];
      const float h = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // half turns
      float s, c;
      sincospif(h, &s, &c);
      cs[buf][angle_at<ADJ>(i)] = make_float2(c, s);
    }
  };
  // token t's positions (lane i: axis i) and place in the caches (lane 0), by warp 0
  auto token = [&](int64_t t, int &pos, int64_t &kv) {
    pos = 0;
    kv = -1;
    if (t >= a.n_tokens) return;
    if (tid < a.num_axes) pos = __ldg(a.positions + (int64_t)tid * a.n_tokens + t);
    if (tid == 0) {
      const int64_t slot = __ldg(a.slot_mapping + t);
      if (slot >= a.num_slots) pa::record_error(a.err, pa::kErrCheck);
      if (slot >= 0 && slot < a.num_slots)
        kv = ((((slot >> a.block_shift) * a.cache_heads) << a.block_shift) +
              (slot & ((1 << a.block_shift) - 1))) *
             (D * (KV8 ? 1 : 2));
    }
  };

  for (int i = tid; i < a.half; i += blockDim.x) {
    int axis = __ldg(a.pair_axis + i);
    if (axis < 0 || axis >= a.num_axes) {
      pa::record_error(a.err, pa::kErrCheck);
      axis = 0;
    }
    s_axis[i] = axis;
    s_turn[i] = __ldg(a.turns + i);
  }
  if (tid < 32) {
    int p0, p1;
    int64_t kv0, kv1;
    token(t, p0, kv0);
    token(t + G, p1, kv1);
    s_pos[0][tid] = p0;
    s_pos[1][tid] = p1;
    if (tid == 0) {
      s_kv[0] = kv0;
      s_kv[1] = kv1;
    }
  }
  __syncthreads();  // (the stages' barriers are initialised, too)
  angles(0);
  __syncthreads();

  volatile int *failed = &s_failed;
  int at = 0;     // of the token in s_kv
  int stage = 0, parity = 0;
  int64_t q_off = t * a.q_out_stride * 2;
  const int64_t q_out_step = G * a.q_out_stride * 2;
  for (int k = 0; t < a.n_tokens; ++k, t += G) {
    const bool more = t + G < a.n_tokens;
    int pos2 = 0;
    int64_t kv2 = -1;
    if (more && tid < 32) token(t + 2 * G, pos2, kv2);
    const int64_t kv = s_kv[at];
    // a wait that gives up is reported, and nothing more is waited for or stored; every
    // thread still comes to every barrier
    bool ok = !*failed;
    if (ok && !pa::mbar_wait_bounded(pa::smem_u32(&s_full[stage]), parity)) {
      pa::record_error(a.err, pa::kErrTimeout);
      *failed = 1;
      ok = false;
    }
    const uint32_t from = stage * stage_bytes;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (!ok || kind[u] == 3 || (kind[u] != 0 && kv < 0)) continue;  // without a slot only q is rotated
      const uint4 x = pa::lds128(src[u] + from + 2 * d0[u]), y = pa::lds128(src[u] + from + 2 * d1[u]);
      float p[8], r[8];
      if (pairs[u] >= 0) {
        if (ADJ) {
          rotate4_adjacent<T>(x, cs[k & 1], pairs[u], p);
          rotate4_adjacent<T>(y, cs[k & 1], d1[u] / 8, r);
        } else {
          rotate8<T>(x, y, cs[k & 1], pairs[u], p, r);
        }
      }
      char *to = dst[u] + (kind[u] == 0 ? q_off : kv);
      if (kind[u] == 0 || !KV8) {
        *reinterpret_cast<uint4 *>(to + 2 * d0[u]) = pairs[u] >= 0 ? narrow8<T>(p) : x;
        *reinterpret_cast<uint4 *>(to + 2 * d1[u]) = pairs[u] >= 0 ? narrow8<T>(r) : y;
      } else {
        if (pairs[u] < 0) {
          widen8<T>(x, p);
          widen8<T>(y, r);
        }
        *reinterpret_cast<uint2 *>(to + d0[u]) = quantise8(p, div[u]);
        *reinterpret_cast<uint2 *>(to + d1[u]) = quantise8(r, div[u]);
      }
    }
    if (!more) break;
    // the next token's angles (its positions were put there an iteration ago); what the
    // one after it needs goes where nobody reads in this iteration
    angles((k + 1) & 1);
    if (tid < 32) s_pos[k & 1][tid] = pos2;
    at = at == 2 ? 0 : at + 1;
    if (tid == 0) s_kv[at == 2 ? 0 : at + 1] = kv2;
    __syncthreads();
    if (tid == 0 && t + a.stages * G < a.n_tokens && !*failed) {
      pa::fence_proxy_async_smem();  // the stage's reads before the copy writes it again
      fetch(t + a.stages * G, stage);
    }
    q_off += q_out_step;
    if (++stage == a.stages) {
      stage = 0;
      parity ^= 1;
    }
  }
  if (*failed && tid == 0)  // copies still in flight land (bounded) before the CTA ends
    for (int i = 0; i < a.stages; ++i)
      for (int b = 0; b < 2; ++b) (void)pa::mbar_wait_bounded(pa::smem_u32(&s_full[i]), b);
}

template <typename T, int D, bool ADJ, bool KV8>
cudaError_t launch_rope(RopeArgs a, cudaStream_t s) {
  auto kern = rope_append_kernel<T, D, ADJ, KV8>;
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int each = (heads * (D / 16) + kPer - 1) / kPer;
  const int threads = (each + 31) / 32 * 32;
  static std::atomic<int> sm_count[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int sms = sm_count[dev].load(std::memory_order_acquire);
  if (sms <= 0) {  // first call on this device: the shared-memory opt-in, too
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMemory);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    sm_count[dev].store(sms, std::memory_order_release);
  }
  // CTAs an SM holds by its threads, and the stages that fit beside each other
  const int bytes = heads * D * 2;
  int ctas = std::max(1, std::min(32, kResident / threads));
  while (ctas > 1 && kStageMemory / ctas / bytes < 2) --ctas;
  a.stages = std::max(2, std::min(kMaxStages, kStageMemory / ctas / bytes));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(a.n_tokens, sms * ctas), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)a.stages * bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, int D>
cudaError_t dispatch_rope(const RopeArgs &a, bool adj, bool kv8, cudaStream_t s) {
  if constexpr (D == 128)
    if (kv8) return adj ? launch_rope<T, D, true, true>(a, s) : launch_rope<T, D, false, true>(a, s);
  if (kv8) return cudaErrorInvalidValue;
  return adj ? launch_rope<T, D, true, false>(a, s) : launch_rope<T, D, false, false>(a, s);
}

}  // namespace

extern "C" PA_API pa_status pa_rope_append(
    void *q_out, const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
    const int32_t *positions, const int64_t *slot_mapping, const int64_t *turns,
    const int32_t *pair_axis, int n_tokens, int num_q_heads, int num_kv_heads, int head_dim,
    int rotary_dim, int num_axes, int interleaved, int64_t q_out_stride, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, int block_size, int num_blocks, pa_dtype dtype,
    const float *k_scale, const float *v_scale, void *stream) {
  if (!q_out || !q || !k || !v || !k_cache || !v_cache || !positions || !slot_mapping || !turns ||
      !pair_axis)
    return PA_ERR_INVALID_ARG;
  if ((k_scale == nullptr) != (v_scale == nullptr)) return PA_ERR_INVALID_ARG;
  if (n_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || rotary_dim <= 0 ||
      num_axes <= 0 || block_size <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  const void *ptrs[6] = {q_out, q, k, v, k_cache, v_cache};
  for (const void *p : ptrs)
    if (!pa::aligned16(p)) return PA_ERR_INVALID_ARG;
  if (!pa::supported_dtype(dtype)) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (k_scale && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (!pa::supported_block(block_size)) return PA_ERR_UNSUPPORTED;
  if (rotary_dim > head_dim) return PA_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (num_q_heads > 65536 || num_kv_heads > 65536) return PA_ERR_INVALID_ARG;
  if (num_axes > kMaxAxes) return PA_ERR_UNSUPPORTED;
  // a token's heads are dense; tokens are any multiple of 16 bytes apart that keeps
  // them from overlapping
  const int64_t wq = (int64_t)num_q_heads * head_dim, wkv = (int64_t)num_kv_heads * head_dim;
  const int64_t strides[4] = {q_out_stride, q_stride, k_stride, v_stride};
  const int64_t widths[4] = {wq, wq, wkv, wkv};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < widths[i] || strides[i] % 8 != 0 || strides[i] > ((int64_t)1 << 40))
      return PA_ERR_INVALID_ARG;
  // (over its own input, each token's rows over themselves)
  if (q_out == q && q_out_stride != q_stride) return PA_ERR_INVALID_ARG;
  if (n_tokens == 0) return PA_OK;
  RopeArgs a;
  a.q_out = static_cast<uint16_t *>(q_out);
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.positions = positions;
  a.slot_mapping = slot_mapping;
  a.turns = turns;
  a.pair_axis = pair_axis;
  a.q_out_stride = q_out_stride;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.num_slots = (int64_t)num_blocks * block_size;
  a.n_tokens = n_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.cache_heads = num_kv_heads;
  a.half = rotary_dim / 2;
  a.num_axes = num_axes;
  a.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.err = pa::error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool kv8 = k_scale != nullptr, adj = interleaved != 0;
  // A launch takes at most kMaxHeads heads of a token (twice as many at head_dim 64), K
  // and V together with as many q heads as fit beside them; usually one does all
  const int most = head_dim == 128 ? kMaxHeads : 2 * kMaxHeads;
  const int kv_step = std::min(num_kv_heads, most / 3);
  const int q_step = most - 2 * kv_step;
  const int launches = std::max((num_q_heads + q_step - 1) / q_step, (num_kv_heads + kv_step - 1) / kv_step);
  for (int i = 0; i < launches; ++i) {
    RopeArgs b = a;
    const int q0 = std::min(num_q_heads, i * q_step), kv0 = std::min(num_kv_heads, i * kv_step);
    b.num_q_heads = std::min(q_step, num_q_heads - q0);
    b.num_kv_heads = std::min(kv_step, num_kv_heads - kv0);
    b.q += (int64_t)q0 * head_dim;
    b.q_out += (int64_t)q0 * head_dim;
    b.k += (int64_t)kv0 * head_dim;
    b.v += (int64_t)kv0 * head_dim;
    const int64_t skip = (int64_t)kv0 * block_size * head_dim * (kv8 ? 1 : 2);
    b.k_cache = static_cast<char *>(k_cache) + skip;
    b.v_cache = static_cast<char *>(v_cache) + skip;
    if (kv8) b.k_scale += kv0, b.v_scale += kv0;
    cudaError_t e;
    if (head_dim == 128)
      e = dtype == PA_FP16 ? dispatch_rope<__half, 128>(b, adj, kv8, s)
                           : dispatch_rope<__nv_bfloat16, 128>(b, adj, kv8, s);
    else
      e = dtype == PA_FP16 ? dispatch_rope<__half, 64>(b, adj, kv8, s)
                           : dispatch_rope<__nv_bfloat16, 64>(b, adj, kv8, s);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}
