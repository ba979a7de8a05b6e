// Decode attention over the 4-bit pool: a warp per query head and quarter of
// the sequence, lanes across the head's elements, fp32 throughout.
#include "decode_fp4.cuh"
#include "pa_fp4.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kWarps = 4;

// N consecutive codes of a row (N = 2, 4 or 8) as floats.
template <int N>
__device__ __forceinline__ void codes_to_floats(const uint8_t* src, float* x) {
  uint32_t w;
  if constexpr (N == 2) w = *src;
  else if constexpr (N == 4) w = *reinterpret_cast<const uint16_t*>(src);
  else w = *reinterpret_cast<const uint32_t*>(src);
  uint32_t h[4];
  e2m1x8_to_half2(w, h);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    x[2 * i] = half_lo(h[i]);
    x[2 * i + 1] = half_hi(h[i]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) decode_fp4_kernel(const Fp4DecodeParams p) {
  constexpr int N = D / 32;
  grid_dependents_launch();
  grid_dependency_wait();
  const int s = blockIdx.y, hq = blockIdx.x, h = hq / p.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = p.seq_lens[s];
  const int BS = 1 << p.log2_block_size;
  if (len > 0 && (((int64_t)len + BS - 1) >> p.log2_block_size) > p.max_blocks_per_seq) {
    if (threadIdx.x == 0) record_error(p.err, PA_DEVERR_SEQ_LEN);
    return;
  }
  const T* q_row = static_cast<const T*>(p.query) + s * p.query_stride + hq * D + lane * N;
  float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = ElemTraits<T>::to_float(q_row[i]) * p.scale_log2;
    o[i] = 0.f;
  }
  const int j = lane * N / kFp4Group, in_group = lane * N % kFp4Group / 2;
  for (int t = warp; t < len; t += kWarps) {
    const int id = p.block_tables[(size_t)s * p.max_blocks_per_seq + (t >> p.log2_block_size)];
    const bool ok = id >= 0 && id < p.num_blocks;
    if (!ok && lane == 0) record_error(p.err, PA_DEVERR_BLOCK_ID);
    const int64_t slot = ((int64_t)(ok ? id : 0) << p.log2_block_size) + (t & (BS - 1));
    const uint8_t* tile =
        p.cache + fp4_tile_offset(slot, h, p.num_kv_heads, p.log2_block_size, D);
    const int row = t & 7;
    float k[N], v[N], x = 0.f;
    codes_to_floats<N>(tile + row * (D / 2) + lane * N / 2, k);
    codes_to_floats<N>(tile + fp4_value_codes(D) + j * 64 + row * 8 + in_group, v);
    const float ks = e4m3_to_float(tile[fp4_key_scales(D) + row * (D / 16) + j]);
    const float vs = e4m3_to_float(tile[fp4_value_scales(D) + j * 8 + row]);
#pragma unroll
    for (int i = 0; i < N; ++i) x = fmaf(q[i], k[i] * ks, x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if (!ok) x = 0.f;
    const float m_new = fmaxf(m, x);
    const float alpha = exp2f(m - m_new), w = exp2f(x - m_new);
    m = m_new;
    l = fmaf(l, alpha, w);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], alpha, ok ? w * (v[i] * vs) : 0.f);
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) so[warp][lane * N + i] = o[i];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float acc = 0.f;
    total = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float a = sl[w] > 0.f || sl[w] != sl[w] ? exp2f(sm[w] - top) : 0.f;
      acc = fmaf(so[w][d], a, acc);
      total = fmaf(sl[w], a, total);
    }
    const float val = len > 0 ? acc / total * p.value_scale : 0.f;
    static_cast<T*>(p.out)[((size_t)s * p.num_heads + hq) * D + d] = ElemTraits<T>::from_float(val);
  }
}

template <typename T, int D>
cudaError_t launch_one(const Fp4DecodeParams& p, cudaStream_t stream) {
  void* args[] = {const_cast<Fp4DecodeParams*>(&p)};
  return launch_overlapped((const void*)decode_fp4_kernel<T, D>,
                           dim3((unsigned)p.num_heads, (unsigned)p.num_seqs), dim3(32 * kWarps), 0,
                           stream, args);
}

}  // namespace

cudaError_t launch_decode_fp4(const Fp4DecodeParams& p, int dtype, int num_sms,
                              cudaStream_t stream) {
  (void)num_sms;
  const bool half = dtype == PA_BF16;
  switch (p.head_size) {
    case 64: return half ? launch_one<__nv_bfloat16, 64>(p, stream) : launch_one<float, 64>(p, stream);
    case 128:
      return half ? launch_one<__nv_bfloat16, 128>(p, stream) : launch_one<float, 128>(p, stream);
    default:
      return half ? launch_one<__nv_bfloat16, 256>(p, stream) : launch_one<float, 256>(p, stream);
  }
}

}  // namespace pa
