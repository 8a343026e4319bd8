// Attention of one new token per sequence over a paged cache (cb_attention_decode):
// the kernel for caches whose rows are not whole 16-byte pieces (the others take
// decode_stream.cuh) and the join of split sequences.
//
// Bound by HBM: every key and value of the batch is read once, and one
// query's 4 FLOP per element are far below the FMA rate until many heads
// share a key head.  decode_common.cuh says how tokens are dealt.
#include "decode_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kThreads = 128;
constexpr int kHeads = kDecodeSimtHeads;

template <typename T>
__global__ void __launch_bounds__(kThreads) decode_simt_kernel(DecodeArgs a) {
  extern __shared__ __align__(16) float smem[];
  const int ldk = (a.dk + 3) / 4 * 4 + 4;
  float* Ks = smem;                           // [64][ldk]
  float* Qs = Ks + kDecodeTile * ldk;         // [kHeads][ldk]
  float* Ps = Qs + kHeads * ldk;              // [64][kHeads]
  float* red = Ps + kDecodeTile * kHeads;     // [kHeads][dv] at the end of a piece
  unsigned* prefix = reinterpret_cast<unsigned*>(red + kHeads * a.dv);
  __shared__ float ms[kHeads], ls[kHeads], corr_s[kHeads];
  __shared__ int page_s[kDecodeTile], slot_s[kDecodeTile];

  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  tile_prefix(a, prefix);
  const int per_seq = a.Hkv * a.chunks;
  const long long total = static_cast<long long>(prefix[a.B]) * per_seq;
  const Run run{total, min(static_cast<long long>(gridDim.x), max(total, 1LL))};
  const long long cta = blockIdx.x;
  if (tid == 0) a.record[2 * cta] = -1;
  zero_empty(a, prefix, [&](long long i) { static_cast<T*>(a.o)[i] = from_f32<T>(0.f); });
  if (cta >= run.ctas || total == 0) return;
  const long long end = run.begin(cta + 1);
  long long at = run.begin(cta);
  int b = find_seq(a, prefix, per_seq, at);
  // threads of one value row: lanes_v of 4 values each
  int lanes_v = 1;
  while (lanes_v * 4 < a.dv) lanes_v <<= 1;
  const int slots = kThreads / lanes_v, vs = tid / lanes_v, vd = (tid % lanes_v) * 4;

  while (at < end) {
    const Piece pc = next_piece(a, prefix, per_seq, at, end, &b);
    const int hk = pc.hk, h0 = pc.h0, heads = pc.heads;

    __syncthreads();
    for (int e = tid; e < kHeads * ldk; e += kThreads) {
      const int g = e / ldk, d = e - g * ldk;
      Qs[e] = g < heads && d < a.dk ? to_f32(static_cast<const T*>(a.q)[b * a.qs_b + (h0 + g) * a.qs_h + d]) : 0.f;
    }
    if (tid < kHeads) ms[tid] = kNegInf, ls[tid] = 0.f;
    float acc[kHeads][4];
#pragma unroll
    for (int g = 0; g < kHeads; ++g)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[g][c] = 0.f;

    for (int t = 0; t < pc.tiles; ++t) {
      const int j0 = (pc.tile0 + t) * kDecodeTile;
      __syncthreads();
      if (tid < kDecodeTile) {
        const int j = j0 + tid;
        page_s[tid] = j >= pc.lo && j < pc.hi ? token_page(a, b, j, &slot_s[tid]) : -1;
      }
      __syncthreads();
      {  // keys
        const int width = ldk - 4;
        for (int e = tid; e < kDecodeTile * width; e += kThreads) {
          const int r = e / width, d = e - r * width;
          const int page = page_s[r];
          Ks[r * ldk + d] = page < 0 || d >= a.dk ? 0.f
                                                  : to_f32(static_cast<const T*>(a.cache.k)[page * a.cache.ks_p + slot_s[r] * a.cache.ks_t + hk * a.cache.ks_h + d]);
        }
      }
      __syncthreads();
      {  // scores: thread = (key, every second head)
        const int key = tid & (kDecodeTile - 1), half = tid >> 6;
        float dot[kHeads / 2];
#pragma unroll
        for (int g = 0; g < kHeads / 2; ++g) dot[g] = 0.f;
        for (int d = 0; d < ldk - 4; d += 4) {
          const float4 kv = *reinterpret_cast<const float4*>(Ks + key * ldk + d);
#pragma unroll
          for (int g = 0; g < kHeads / 2; ++g) {
            const float4 qv = *reinterpret_cast<const float4*>(Qs + (2 * g + half) * ldk + d);
            dot[g] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, dot[g]))));
          }
        }
        const int dist = pc.len - 1 - (j0 + key);
#pragma unroll
        for (int g = 0; g < kHeads / 2; ++g) {
          const int hd = 2 * g + half;
          float x = dot[g] * a.scale;
          if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
          const float slope = a.slopes && hd < heads ? a.slopes[h0 + hd] * kLog2e : 0.f;
          Ps[key * kHeads + hd] = page_s[key] < 0 ? kNegInf : fmaf(-slope, static_cast<float>(dist), x * kLog2e);
        }
      }
      __syncthreads();
      for (int g = warp; g < heads; g += kThreads / 32) {
        const float x0 = Ps[lane * kHeads + g], x1 = Ps[(lane + 32) * kHeads + g];
        float mx = fmaxf(x0, x1);
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
        const float m = ms[g], mn = fmaxf(m, mx), mu = mn == kNegInf ? 0.f : mn;
        const float p0 = exp2_approx(x0 - mu), p1 = exp2_approx(x1 - mu);
        float sum = p0 + p1;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        Ps[lane * kHeads + g] = p0;
        Ps[(lane + 32) * kHeads + g] = p1;
        __syncwarp();
        if (lane == 0) {
          const float corr = exp2_approx(m - mu);
          corr_s[g] = corr;
          ms[g] = mn;
          ls[g] = ls[g] * corr + sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        const float corr = g < heads ? corr_s[g] : 1.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[g][c] *= corr;
      }
      if (vd < a.dv) {
        for (int key = vs; key < kDecodeTile; key += slots) {
          const int page = page_s[key];
          if (page < 0) continue;
          const T* src = static_cast<const T*>(a.cache.v) + page * a.cache.vs_p + slot_s[key] * a.cache.vs_t + hk * a.cache.vs_h + vd;
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = vd + c < a.dv ? to_f32(src[c]) : 0.f;
          const float4 pa = *reinterpret_cast<const float4*>(Ps + key * kHeads);
          const float4 pb = *reinterpret_cast<const float4*>(Ps + key * kHeads + 4);
          const float p[kHeads] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
          for (int g = 0; g < kHeads; ++g)
            if (g < heads)
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[g][c] = fmaf(p[g], v[c], acc[g][c]);
        }
      }
    }
    // The value slots' sums, in slot order.
    for (int s = 0; s < slots; ++s) {
      __syncthreads();
      if (vs == s) {
#pragma unroll
        for (int g = 0; g < kHeads; ++g)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (vd + c < a.dv) red[g * a.dv + vd + c] = (s ? red[g * a.dv + vd + c] : 0.f) + acc[g][c];
      }
    }
    __syncthreads();
    if (pc.starts && pc.ends) {
      for (int e = tid; e < heads * a.dv; e += kThreads) {
        const int g = e / a.dv, d = e - g * a.dv;
        static_cast<T*>(a.o)[b * a.os_b + (h0 + g) * a.os_h + d] = from_f32<T>(ls[g] == 0.f ? 0.f : red[e] / ls[g]);
      }
    } else {
      float* part = a.part + (2 * cta + (pc.starts ? 1 : 0)) * part_floats(a.item_heads, a.dv);
      for (int e = tid; e < heads * a.dv; e += kThreads) part[2 * a.item_heads + e] = red[e];
      if (tid < heads) part[tid] = ms[tid], part[a.item_heads + tid] = ls[tid];
      if (pc.starts && tid == 0) note_item(a, run, pc, per_seq, cta);
    }
    at += pc.dealt;
  }
}

// One item that several CTAs shared: the CTA that holds its start (slot 1)
// and the ones after it (slot 0).  out = sum w o / sum w l, w = 2^(m - max m).
template <typename T>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeArgs a) {
  __shared__ __align__(16) float sum_s[8][128];
  __shared__ float l_s[8];
  pdl_wait();
  pdl_launch_dependents();
  const int cta = blockIdx.x;
  const int rec = a.record[2 * cta], pieces = a.record[2 * cta + 1];
  if (rec < 0) return;
  const int per_seq = a.Hkv * a.chunks;
  const int b = rec / per_seq, item = rec - b * per_seq;
  const int hk = item / a.chunks, h0 = hk * a.group + (item % a.chunks) * a.item_heads;
  const int heads = min(a.item_heads, (hk + 1) * a.group - h0), g = blockIdx.y;
  if (g >= heads) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t pf = part_floats(a.item_heads, a.dv);
  auto part = [&](int i) { return a.part + (i == 0 ? 2 * static_cast<size_t>(cta) + 1 : 2 * (static_cast<size_t>(cta) + i)) * pf; };
  float m = kNegInf;
  for (int i = lane; i < pieces; i += 32) m = fmaxf(m, part(i)[g]);
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const float mu = m == kNegInf ? 0.f : m;
  float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = warp; i < pieces; i += 8) {
    const float* p = part(i);
    const float w = exp2_approx(p[g] - mu);
    l = fmaf(w, p[a.item_heads + g], l);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < a.dv) acc[c] = fmaf(w, p[2 * a.item_heads + g * a.dv + lane + 32 * c], acc[c]);
  }
  for (int c = 0; c < 4; ++c) sum_s[warp][lane + 32 * c] = acc[c];
  if (lane == 0) l_s[warp] = l;
  __syncthreads();
  if (threadIdx.x < a.dv) {
    float o = 0.f, ll = 0.f;
    for (int w = 0; w < 8; ++w) o += sum_s[w][threadIdx.x], ll += l_s[w];
    static_cast<T*>(a.o)[b * a.os_b + (h0 + g) * a.os_h + threadIdx.x] = from_f32<T>(ll == 0.f ? 0.f : o / ll);
  }
}

size_t simt_smem(int dk, int dv, int B) {
  const size_t ldk = (dk + 3) / 4 * 4 + 4;
  return sizeof(float) * ((kDecodeTile + kHeads) * ldk + kDecodeTile * kHeads + static_cast<size_t>(kHeads) * dv) +
         sizeof(unsigned) * (B + 1);
}

template <typename T>
cudaError_t launch_simt(const DecodeArgs& a, cudaStream_t s) {
  const size_t smem = simt_smem(a.dk, a.dv, a.B);
  const cudaError_t e = smem_attr_once<decode_simt_kernel<T>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_simt_kernel<T>, dim3(a.ctas), dim3(kThreads), smem, s, a);
}

template <typename T>
cudaError_t launch_join(const DecodeArgs& a, cudaStream_t s) {
  return launch_pdl(decode_join_kernel<T>, dim3(a.ctas, a.item_heads), dim3(256), 0, s, a);
}

}  // namespace

size_t decode_workspace_bytes(int ctas, int heads, int dv) {
  return sizeof(float) * 2 * ctas * part_floats(heads, dv) + sizeof(int) * 2 * ctas;
}

cudaError_t launch_attn_rows(const AttnArgs& rw, bool bf16, int sms, cudaStream_t s) {
  DecodeArgs a{};
  a.scale = rw.scale, a.softcap = rw.softcap;
  a.B = rw.B, a.Hq = rw.Hq, a.group = rw.group, a.Hkv = rw.Hq / rw.group;
  a.dk = rw.dk, a.dv = rw.dv;
  // a sequence is one page of Lk slots
  a.cache.k = const_cast<void*>(rw.k), a.cache.v = const_cast<void*>(rw.v);
  a.cache.ks_p = rw.ks_b, a.cache.ks_t = rw.ks_l, a.cache.ks_h = rw.ks_h;
  a.cache.vs_p = rw.vs_b, a.cache.vs_t = rw.vs_l, a.cache.vs_h = rw.vs_h;
  const int rows = rw.Lq * rw.group, most = bf16 ? kDecodeMmaHeads : kDecodeSimtHeads;
  a.chunks = (rows + most - 1) / most;
  a.item_heads = (rows + a.chunks - 1) / a.chunks;
  // A cluster per item while that fills the GPU better and leaves every CTA a tile.
  const long long items = static_cast<long long>(a.B) * a.Hkv * a.chunks, room = sms * decode_ctas_per_sm(a.dk, a.dv, bf16, a.item_heads, 0);
  const int tiles = (rw.Lk + 63) / 64;
  a.split = 1;
  while (a.split < 8 && items * a.split * 2 <= room && a.split < tiles) a.split *= 2;
  return bf16 ? launch_rows_mma(a, rw, s) : launch_rows_fma(a, rw, s);
}

cudaError_t launch_decode(const DecodeArgs& a, bool bf16, bool vec, cudaStream_t s) {
  cudaError_t e;
  if (vec)
    e = bf16 ? launch_decode_mma(a, s) : launch_decode_fma(a, s);
  else
    e = bf16 ? launch_simt<__nv_bfloat16>(a, s) : launch_simt<float>(a, s);
  if (e != cudaSuccess || a.split) return e;
  return bf16 ? launch_join<__nv_bfloat16>(a, s) : launch_join<float>(a, s);
}

}  // namespace cb
