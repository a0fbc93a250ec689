// pa_scored_prefill.cu -- host launchers of the many-row tensor-core kernel that also
// writes each row's statistics (scored attention), both element types.
#include "pa_prefill_inst.cuh"

namespace pa {

cudaError_t launch_prefill_stats(const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const CUtensorMap &qmap, const DecodeArgs &args, int head_dim,
                                 bool fp16, bool kv8, cudaStream_t stream) {
  if (args.block_size == 16)
    return fp16 ? dispatch_stats<true, __half>(kmap, vmap, qmap, args, head_dim, kv8, stream)
                : dispatch_stats<true, __nv_bfloat16>(kmap, vmap, qmap, args, head_dim, kv8, stream);
  return fp16 ? dispatch_stats<false, __half>(kmap, vmap, qmap, args, head_dim, kv8, stream)
              : dispatch_stats<false, __nv_bfloat16>(kmap, vmap, qmap, args, head_dim, kv8, stream);
}

}  // namespace pa
