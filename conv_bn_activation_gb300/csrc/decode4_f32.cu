// Attention over a 4-bit cache with fp32 queries (decode4.cuh).
#include "decode4.cuh"

namespace cb {

cudaError_t launch_decode4_f32(const DecodeArgs& a, const Units4& u, const Maps4* maps, cudaStream_t s) {
  return decode4_dim(a.dk, a.dv) == 64 ? launch_decode4_shape<Decode4Shape<64, 64, 1, float>>(a, u, maps, s)
                                       : launch_decode4_shape<Decode4Shape<128, 128, 1, float>>(a, u, maps, s);
}

}  // namespace cb
