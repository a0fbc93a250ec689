// pa_block_scaled.cu -- the quantising append of a block-scaled FP8 cache.
//
// A block's rows of one KV head share one scale for K and one for V:
//   need = the least power of two with  max |x| <= 448 need  over the new rows' finite x
//   s    = need                     where the block's first row is new
//        = max(s_old, need)         where rows stand before the new ones
//   new rows:    code = e4m3(x / s)
//   older rows, where s grew:  code = e4m3(code * s_old / s)
// A power of two costs an e4m3 value no precision (only the exponent moves), makes x / s
// a multiplication without rounding, and an older row is rounded again only where its
// codes become subnormal.  The least power of two is read off the bits of the maximum:
// 448 = 1.75 * 2^8.
//
// Bound by memory: two bytes read and one written an element.  One warp takes the rows of
// one (block, KV head) of K or of V: it holds the new rows in registers (16 of 16 tokens:
// 32 registers a lane) between the maximum and the rounding, so they are read once, with
// every 16-byte load under way before the first use.  16 x 512 tokens of 32 heads take 35.1 us,
// 5.75 TB/s or 0.85 of a plain copy's rate; one token of 64 sequences and 8 heads 7.0 with the
// call, a chain of dependent loads (length, table, scale).
#include <algorithm>

#include "../../include/pagedattn.h"
#include "pa_decode.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace pa {
namespace {

struct AppendArgs {
  uint8_t *cache[2];
  float *kv_scales;
  const uint16_t *rows[2];
  int64_t stride[2];
  const int32_t *block_tables, *context_lens;
  int num_seqs, q_len, num_kv_heads, max_blocks_per_seq, num_blocks;
  int touched;  // blocks that q_len positions can touch
  unsigned *err;
};

// The least power of two s with top <= 448 s, within the range of block scales.
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t b = __float_as_uint(top);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, -40), 40);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Eight 16-bit values times f (a power of two) -> eight e4m3 codes.
template <typename T>
__device__ __forceinline__ uint2 codes_of(const uint4 v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = Elt<T>::to_f2(w[i]);
    c[i] = f32x2_to_e4m3x2(x.x * f, x.y * f);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <typename T, int BSZ>
__global__ void __launch_bounds__(128) append_block_scaled_kernel(const AppendArgs a) {
  constexpr int D = 128;
  constexpr int kLoads = BSZ / 2;  // two rows a load: 16 lanes of 16 bytes each
  constexpr uint32_t kInf = Elt<T>::kMantBits == 10 ? 0x7c00u : 0x7f80u;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  // (KV head fastest: neighbouring warps read neighbouring parts of the tokens)
  int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = (int)(unit % a.num_kv_heads);
  unit /= a.num_kv_heads;
  const int kv = (int)(unit & 1);
  unit >>= 1;
  const int t = (int)(unit % a.touched);
  const int64_t seq = unit / a.touched;
  if (seq >= a.num_seqs) return;
  const int L = max(0, __ldg(a.context_lens + seq));
  const int64_t first = (int64_t)L - a.q_len;  // position of the sequence's new row 0
  const int lb = (int)(first > 0 ? first / BSZ : 0) + t;
  const int64_t pos0 = (int64_t)lb * BSZ;
  if (pos0 >= L) return;
  int blk = -1;
  if (lb < a.max_blocks_per_seq) blk = __ldg(a.block_tables + seq * a.max_blocks_per_seq + lb);
  if (blk < 0 || blk >= a.num_blocks) {
    if (lane == 0) record_error(a.err, kErrCheck);
    return;
  }
  const int r0 = first > pos0 ? (int)(first - pos0) : 0;            // new rows [r0, r1)
  const int r1 = (int)(L - pos0 < BSZ ? L - pos0 : BSZ);

  // the old scale, and the new rows: lane l holds chunk l % 16 of rows l / 16, + 2, ..
  float *sp = a.kv_scales + ((int64_t)blk * a.num_kv_heads + h) * 2 + kv;
  const float s_old = r0 > 0 ? clamp_scale(__ldcg(sp)) : 0.f;
  const int half = lane >> 4, ch = lane & 15;
  const uint16_t *src = a.rows[kv] + (seq * a.q_len + (pos0 - first)) * a.stride[kv] + (int64_t)h * D + ch * 8;
  uint4 x[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int r = 2 * k + half;
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= r0 && r < r1) x[k] = __ldg(reinterpret_cast<const uint4 *>(src + r * a.stride[kv]));
  }
  // magnitudes as integers order as the values do
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    m = __vmaxu2(m, x[k].x & 0x7fff7fffu);
    m = __vmaxu2(m, x[k].y & 0x7fff7fffu);
    m = __vmaxu2(m, x[k].z & 0x7fff7fffu);
    m = __vmaxu2(m, x[k].w & 0x7fff7fffu);
  }
  uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if (top >= kInf) {  // infinities and NaN do not count
    top = 0u;
#pragma unroll 1
    for (int k = 0; k < kLoads; ++k) {
      uint4 v = x[0];
#pragma unroll
      for (int i = 1; i < kLoads; ++i) v = i == k ? x[i] : v;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        top = max(top, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const float need = scale_for(Elt<T>::to_f2(top).x);
  const float s = r0 > 0 ? fmaxf(s_old, need) : need;

  uint8_t *page = a.cache[kv] + ((int64_t)blk * a.num_kv_heads + h) * (BSZ * D);
  if (r0 > 0 && s > s_old) {  // older rows to the new scale: 4 rows a step, 8 lanes each
    const float f = s_old / s;
    for (int r = lane >> 3; r < r0; r += 4) {
      uint4 *p = reinterpret_cast<uint4 *>(page + r * D) + (lane & 7);
      float v[16];
      e4m3x16_to_f32(__ldcg(p), v);
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = f32x2_to_e4m3x2(v[2 * i] * f, v[2 * i + 1] * f);
      *p = make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16), c[6] | (c[7] << 16));
    }
  }
  // x / s: s is a power of two, unless a foreign cache's scale stands
  const bool exact = (__float_as_uint(s) & 0x7fffffu) == 0u;
  const float inv = 1.f / s;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int r = 2 * k + half;
    if (r >= r0 && r < r1)
      reinterpret_cast<uint2 *>(page + r * D)[ch] = exact ? codes_of<T>(x[k], inv) : quantize8<T>(x[k], s);
  }
  if (lane == 0) *sp = s;
}

template <typename T>
cudaError_t launch_append(const AppendArgs &a, int block_size, cudaStream_t st) {
  const int64_t warps = (int64_t)a.num_seqs * a.touched * 2 * a.num_kv_heads;
  const int64_t ctas = (warps + 3) / 4;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)ctas);
  if (block_size == 8) return launch_dependent(append_block_scaled_kernel<T, 8>, grid, 128, st, a);
  if (block_size == 16) return launch_dependent(append_block_scaled_kernel<T, 16>, grid, 128, st, a);
  return launch_dependent(append_block_scaled_kernel<T, 32>, grid, 128, st, a);
}

}  // namespace
}  // namespace pa

extern "C" PA_API pa_status pa_append_kv_block_scaled(
    void *k_cache, void *v_cache, float *kv_scales, const void *k_new, const void *v_new,
    const int32_t *block_tables, const int32_t *context_lens, int num_seqs, int num_kv_heads, int head_dim,
    int block_size, int max_blocks_per_seq, int num_blocks, int q_len, pa_dtype new_dtype, int64_t k_stride,
    int64_t v_stride, void *stream) {
  using namespace pa;
  if (!k_cache || !v_cache || !kv_scales || !k_new || !v_new || !block_tables || !context_lens)
    return PA_ERR_INVALID_ARG;
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0 || q_len <= 0)
    return PA_ERR_INVALID_ARG;
  for (const void *p : {static_cast<const void *>(k_cache), static_cast<const void *>(v_cache),
                        static_cast<const void *>(kv_scales), k_new, v_new})
    if (!aligned16(p)) return PA_ERR_INVALID_ARG;
  if (!aligned4(block_tables) || !aligned4(context_lens)) return PA_ERR_INVALID_ARG;
  if (!supported_dtype(new_dtype)) return PA_ERR_UNSUPPORTED;
  if (head_dim != 128 || !supported_block(block_size) || q_len > 4096) return PA_ERR_UNSUPPORTED;
  const int64_t width = (int64_t)num_kv_heads * head_dim;
  for (const int64_t st : {k_stride, v_stride})
    if (st < width || st % 8 != 0 || st >= (int64_t)1 << 40) return PA_ERR_INVALID_ARG;
  if ((int64_t)num_blocks * num_kv_heads * 2 >= (int64_t)1 << 31 ||
      (int64_t)num_seqs * max_blocks_per_seq * 2 >= (int64_t)1 << 31 ||
      (int64_t)max_blocks_per_seq * block_size >= (int64_t)1 << 31 ||
      (int64_t)num_seqs * q_len * num_kv_heads >= (int64_t)1 << 31)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  const int64_t tokens = (int64_t)num_seqs * q_len;
  for (const int64_t st : {k_stride, v_stride})
    if (st > ((int64_t)1 << 58) / tokens) return PA_ERR_INVALID_ARG;  // (past every address)
  // the caches and their scales apart from one another and from what is read (k_new and v_new may
  // be slices of one array)
  const size_t cache = (size_t)num_blocks * num_kv_heads * block_size * head_dim;
  struct {
    const void *p;
    size_t n;
  } buf[] = {{k_cache, cache}, {v_cache, cache}, {kv_scales, (size_t)num_blocks * num_kv_heads * 8},
             {k_new, (size_t)((tokens - 1) * k_stride + width) * 2},
             {v_new, (size_t)((tokens - 1) * v_stride + width) * 2},
             {block_tables, (size_t)num_seqs * max_blocks_per_seq * 4}, {context_lens, (size_t)num_seqs * 4}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 7; ++j)
      if (overlap(buf[i].p, buf[i].n, buf[j].p, buf[j].n)) return PA_ERR_INVALID_ARG;
  AppendArgs a;
  a.cache[0] = static_cast<uint8_t *>(k_cache);
  a.cache[1] = static_cast<uint8_t *>(v_cache);
  a.kv_scales = kv_scales;
  a.rows[0] = static_cast<const uint16_t *>(k_new);
  a.rows[1] = static_cast<const uint16_t *>(v_new);
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.num_seqs = num_seqs;
  a.q_len = q_len;
  a.num_kv_heads = num_kv_heads;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.touched = (q_len + block_size - 2) / block_size + 1;
  a.err = error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = new_dtype == PA_FP16 ? launch_append<__half>(a, block_size, s)
                                             : launch_append<__nv_bfloat16>(a, block_size, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
