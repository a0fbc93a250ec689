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
#include <cuda_runtime.h>

#include <algorithm>

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
  int n_tokens, num_q_heads, num_kv_heads, half, num_axes, block_size;
  const float *k_scale, *v_scale;
  unsigned *err;
};

// Eight rotated pairs: a (16 bytes of first elements) and b (of second elements),
// cs[0..7] their (cos, sin); fp32 results in x (a') and y (b').
template <typename T>
__device__ __forceinline__ void rotate8(const uint4 a, const uint4 b, const float2 *cs,
                                        float (&x)[8], float (&y)[8]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 fa = pa::Elt<T>::to_f2(wa[i]), fb = pa::Elt<T>::to_f2(wb[i]);
    const float4 c = *reinterpret_cast<const float4 *>(cs + 2 * i);  // cos, sin of two pairs
    x[2 * i] = fmaf(fa.x, c.x, -fb.x * c.y);
    y[2 * i] = fmaf(fb.x, c.x, fa.x * c.y);
    x[2 * i + 1] = fmaf(fa.y, c.z, -fb.y * c.w);
    y[2 * i + 1] = fmaf(fb.y, c.z, fa.y * c.w);
  }
}

// Eight adjacent pairs in 32 bytes a, b: the same with the pairs' elements adjacent;
// x holds the results for a's elements, y for b's.
template <typename T>
__device__ __forceinline__ void rotate8_adjacent(const uint4 a, const uint4 b, const float2 *cs,
                                                 float (&x)[8], float (&y)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = pa::Elt<T>::to_f2(w[i]);
    const float2 c = cs[i];
    float *o = i < 4 ? x + 2 * i : y + 2 * (i - 4);
    o[0] = fmaf(f.x, c.x, -f.y * c.y);
    o[1] = fmaf(f.y, c.x, f.x * c.y);
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

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = pa::f32x2_to_e4m3x2(x[2 * i] / scale, x[2 * i + 1] / scale);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

constexpr int kMaxHalf = 64;  // rotary pairs per head at most (head_dim 128)

// CTA t takes token t.  An item is 16 elements of one head: the two 16-byte chunks
// of eight rotated pairs, or two adjacent chunks that are copied (V, and elements
// past rotary_dim).  Heads are numbered q, then K, then V.
template <typename T, int D, bool ADJ, bool KV8>
__global__ void rope_append_kernel(const RopeArgs a) {
  constexpr int kItems = D / 16;  // items of a head
  __shared__ __align__(16) float2 cs[kMaxHalf];
  pa::griddep_wait();
  pa::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  for (int i = threadIdx.x; i < a.half; i += blockDim.x) {
    int axis = __ldg(a.pair_axis + i);
    if (axis < 0 || axis >= a.num_axes) {
      pa::record_error(a.err, pa::kErrCheck);
      axis = 0;
    }
    const int64_t pos = __ldg(a.positions + (int64_t)axis * a.n_tokens + t);
    const uint64_t turn = (uint64_t)pos * (uint64_t)__ldg(a.turns + i);
    const float h = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // half turns
    float s, c;
    sincospif(h, &s, &c);
    cs[i] = make_float2(c, s);
  }
  int64_t blk = -1;
  int off = 0;
  const int64_t slot = __ldg(a.slot_mapping + t);
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0) pa::record_error(a.err, pa::kErrCheck);
  } else if (slot >= 0) {
    blk = slot / a.block_size;
    off = (int)(slot - blk * a.block_size);
  }
  __syncthreads();

  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int rot_items = a.half / 8;
  const int heads = blk < 0 ? hq : hq + 2 * hkv;  // without a slot only q is rotated
  for (int it = threadIdx.x; it < heads * kItems; it += blockDim.x) {
    const int h = it / kItems, c = it % kItems;
    const bool is_q = h < hq, is_k = !is_q && h < hq + hkv;
    const uint16_t *src = is_q ? a.q + t * a.q_stride + (int64_t)h * D
                         : is_k ? a.k + t * a.k_stride + (int64_t)(h - hq) * D
                                : a.v + t * a.v_stride + (int64_t)(h - hq - hkv) * D;
    const bool rot = (is_q || is_k) && c < rot_items;
    const int e0 = (rot && !ADJ) ? 8 * c : 16 * c;
    const int e1 = (rot && !ADJ) ? 8 * c + a.half : 16 * c + 8;
    const uint4 u0 = *reinterpret_cast<const uint4 *>(src + e0);
    const uint4 u1 = *reinterpret_cast<const uint4 *>(src + e1);
    float x[8], y[8];
    if (rot) {
      if (ADJ)
        rotate8_adjacent<T>(u0, u1, cs + 8 * c, x, y);
      else
        rotate8<T>(u0, u1, cs + 8 * c, x, y);
    }
    if (is_q) {
      uint16_t *dst = a.q_out + t * a.q_out_stride + (int64_t)h * D;
      *reinterpret_cast<uint4 *>(dst + e0) = rot ? narrow8<T>(x) : u0;
      *reinterpret_cast<uint4 *>(dst + e1) = rot ? narrow8<T>(y) : u1;
    } else {
      const int hh = is_k ? h - hq : h - hq - hkv;
      const int64_t row = ((blk * hkv + hh) * a.block_size + off) * D;
      void *cache = is_k ? a.k_cache : a.v_cache;
      if constexpr (KV8) {
        if (!rot) {
          widen8<T>(u0, x);
          widen8<T>(u1, y);
        }
        const float scale = __ldg((is_k ? a.k_scale : a.v_scale) + hh);
        uint8_t *dst = static_cast<uint8_t *>(cache) + row;
        *reinterpret_cast<uint2 *>(dst + e0) = quantise8(x, scale);
        *reinterpret_cast<uint2 *>(dst + e1) = quantise8(y, scale);
      } else {
        uint16_t *dst = static_cast<uint16_t *>(cache) + row;
        *reinterpret_cast<uint4 *>(dst + e0) = rot ? narrow8<T>(x) : u0;
        *reinterpret_cast<uint4 *>(dst + e1) = rot ? narrow8<T>(y) : u1;
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_rope(const RopeArgs &a, bool adj, bool kv8, cudaStream_t s) {
  const int items = (a.num_q_heads + 2 * a.num_kv_heads) * (D / 16);
  const unsigned threads = (unsigned)std::min(256, (items + 31) / 32 * 32);
  const dim3 grid((unsigned)a.n_tokens, 1, 1);
  if (kv8) {
    if constexpr (D == 128)
      return adj ? pa::launch_dependent(rope_append_kernel<T, D, true, true>, grid, threads, s, a)
                 : pa::launch_dependent(rope_append_kernel<T, D, false, true>, grid, threads, s, a);
    return cudaErrorInvalidValue;
  }
  return adj ? pa::launch_dependent(rope_append_kernel<T, D, true, false>, grid, threads, s, a)
             : pa::launch_dependent(rope_append_kernel<T, D, false, false>, grid, threads, s, a);
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
  // a token's heads are dense; tokens are any multiple of 16 bytes apart that keeps
  // them from overlapping
  const int64_t wq = (int64_t)num_q_heads * head_dim, wkv = (int64_t)num_kv_heads * head_dim;
  const int64_t strides[4] = {q_out_stride, q_stride, k_stride, v_stride};
  const int64_t widths[4] = {wq, wq, wkv, wkv};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < widths[i] || strides[i] % 8 != 0 || strides[i] > ((int64_t)1 << 40))
      return PA_ERR_INVALID_ARG;
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
  a.half = rotary_dim / 2;
  a.num_axes = num_axes;
  a.block_size = block_size;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.err = pa::error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool kv8 = k_scale != nullptr, adj = interleaved != 0;
  cudaError_t e;
  if (head_dim == 128)
    e = dtype == PA_FP16 ? launch_rope<__half, 128>(a, adj, kv8, s)
                         : launch_rope<__nv_bfloat16, 128>(a, adj, kv8, s);
  else
    e = dtype == PA_FP16 ? launch_rope<__half, 64>(a, adj, kv8, s)
                         : launch_rope<__nv_bfloat16, 64>(a, adj, kv8, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
