// pa_block_scaled_fp16.cu -- fp16 instantiations of the decode kernels over a block-scaled FP8
// cache, for all block sizes.
#include "pa_decode_inst.cuh"

namespace pa {
cudaError_t launch_decode8b_fp16(const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const DecodeArgs &args, bool partial, int units, cudaStream_t stream) {
  using T = __half;
  return args.block_size == 16 ? launch_decode8_t<16, T, false, true>(kmap, vmap, args, partial, units, stream)
                               : launch_decode8_t<0, T, false, true>(kmap, vmap, args, partial, units, stream);
}
}  // namespace pa
