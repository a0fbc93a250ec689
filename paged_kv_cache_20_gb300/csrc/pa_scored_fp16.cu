// pa_scored_fp16.cu -- fp16 instantiations of the decode kernels that also write every
// score (scored decode), for all block sizes.
#include "pa_decode_inst.cuh"

namespace pa {
cudaError_t launch_decode_scored_fp16(const CUtensorMap &kmap, const CUtensorMap &vmap,
                                      const DecodeArgs &args, int head_dim, bool kv8, bool partial,
                                      int units, cudaStream_t stream) {
  using T = __half;
  if (kv8)
    return args.block_size == 16
               ? launch_decode8_t<16, T, true>(kmap, vmap, args, partial, units, stream)
               : launch_decode8_t<0, T, true>(kmap, vmap, args, partial, units, stream);
  return args.block_size == 16
             ? launch_decode_t<16, T, true>(kmap, vmap, args, head_dim, partial, units, stream)
             : launch_decode_t<0, T, true>(kmap, vmap, args, head_dim, partial, units, stream);
}
}  // namespace pa
