// pa_block_scaled_prefill.cu -- host launcher of the many-row tensor-core kernel over a
// block-scaled FP8 cache, both element types, all block sizes.
#include "pa_prefill_inst.cuh"

namespace pa {

namespace {
template <bool BS16, typename T>
cudaError_t launch_scaled(const CUtensorMap &kmap, const CUtensorMap &vmap, const CUtensorMap &qmap,
                          const DecodeArgs &a, bool partial, cudaStream_t st) {
  return partial ? launch_prefill_t<T, 128, true, true, BS16, false, true>(kmap, vmap, qmap, a, st)
                 : launch_prefill_t<T, 128, false, true, BS16, false, true>(kmap, vmap, qmap, a, st);
}
}  // namespace

cudaError_t launch_prefill8b(const CUtensorMap &kmap, const CUtensorMap &vmap, const CUtensorMap &qmap,
                             const DecodeArgs &a, bool fp16, bool partial, cudaStream_t st) {
  if (a.block_size == 16)
    return fp16 ? launch_scaled<true, __half>(kmap, vmap, qmap, a, partial, st)
                : launch_scaled<true, __nv_bfloat16>(kmap, vmap, qmap, a, partial, st);
  return fp16 ? launch_scaled<false, __half>(kmap, vmap, qmap, a, partial, st)
              : launch_scaled<false, __nv_bfloat16>(kmap, vmap, qmap, a, partial, st);
}

}  // namespace pa
