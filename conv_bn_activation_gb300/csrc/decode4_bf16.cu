// Attention over a 4-bit cache with bf16 queries (decode4.cuh).  One shape of the
// kernel serves keys and values up to 64 dims, another those up to 128: what a
// row lacks is not copied.
#include "decode4.cuh"

namespace cb {

namespace {

template <int D>
cudaError_t launch_dims(const DecodeArgs& a, const Units4& u, const Maps4* maps, cudaStream_t s) {
  return a.item_heads <= 8 ? launch_decode4_shape<Decode4Shape<D, D, 1, __nv_bfloat16>>(a, u, maps, s)
                           : launch_decode4_shape<Decode4Shape<D, D, 2, __nv_bfloat16>>(a, u, maps, s);
}

}  // namespace

cudaError_t launch_decode4_bf16(const DecodeArgs& a, const Units4& u, const Maps4* maps, cudaStream_t s) {
  return decode4_dim(a.dk, a.dv) == 64 ? launch_dims<64>(a, u, maps, s) : launch_dims<128>(a, u, maps, s);
}

}  // namespace cb
