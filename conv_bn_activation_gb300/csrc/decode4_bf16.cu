// Attention over a 4-bit cache with bf16 queries (decode4.cuh).
#include "decode4.cuh"

namespace cb {

namespace {

template <int DK, int DV>
cudaError_t launch_dims(const DecodeArgs& a, const Units4& u, const Maps4* maps, cudaStream_t s) {
  return a.item_heads <= 8 ? launch_decode4_shape<Decode4Shape<DK, DV, 1, __nv_bfloat16>>(a, u, maps, s)
                           : launch_decode4_shape<Decode4Shape<DK, DV, 2, __nv_bfloat16>>(a, u, maps, s);
}

}  // namespace

cudaError_t launch_decode4_bf16(const DecodeArgs& a, const Units4& u, const Maps4* maps, cudaStream_t s) {
  if (a.dk <= 64) return a.dv <= 64 ? launch_dims<64, 64>(a, u, maps, s) : launch_dims<64, 128>(a, u, maps, s);
  return a.dv <= 64 ? launch_dims<128, 64>(a, u, maps, s) : launch_dims<128, 128>(a, u, maps, s);
}

}  // namespace cb
