// Norms of queries and keys for each head, and the rotation by position, in one pass for
// sm_103a (pa_norm_rope).
//
// Every element is read once and written once; memory bounds it.  A head's row goes over
// D / 16 lanes, 16 elements each, which are eight pairs: the lane's two groups of eight
// neighbours are the pairs' first and second elements (halves), or the pairs lie inside the
// groups (neighbours).  Either way the lane's cosines and sines are eight in a row of the
// table, and no element leaves its lane.  A token's heads are shared out over lanes that go
// through them with the same cosines.
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  pa_norm_rope_args a;
  unsigned int* err;
  int groups;  // rows of lanes that share a token's heads
};

// Eight elements as fp32, and back.
template <typename T>
struct Eight {
  static constexpr int kVecs = sizeof(T) / 2;
  uint4 w[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void unpack(float* x) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) ElemTraits<T>::unpack(w[i], x + i * ElemTraits<T>::kPerChunk);
  }
  static __device__ __forceinline__ void store(T* p, const float* x) {
    if constexpr (sizeof(T) == 2) {
      stg_v4(p, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                           pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        stg_v4(p + 4 * i, make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                     __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3])));
    }
  }
};

// A thread has 16 elements of each of N heads of a token, all of which it asks for at
// once, and before it knows the position.
template <typename T, int D, int N>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;  // of a row
  const pa_norm_rope_args& a = p.a;
  const int64_t unit = (int64_t)blockIdx.x * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
  const int j = threadIdx.x % kLanes;
  const int64_t t = unit / p.groups;
  const int first = (int)(unit - t * p.groups);
  const int half = a.rotary_dim / 16;  // lanes that rotate
  const bool turns = j < half;
  // The lane's two groups of eight.
  const int g0 = a.interleaved || !turns ? 2 * j : j;
  const int g1 = a.interleaved || !turns ? 2 * j + 1 : j + half;
  const int heads = a.num_heads + a.num_kv_heads;
  grid_dependents_launch();
  grid_dependency_wait();
  // Lanes of other tokens share the warp: they come along to its shuffles.
  bool live = t < a.num_tokens;
  Eight<T> w[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = first + i * p.groups;
    if (live && h < heads) {
      const T* src = h < a.num_heads
                         ? static_cast<const T*>(a.query) + t * a.query_stride + h * D
                         : static_cast<const T*>(a.key) + t * a.key_stride + (h - a.num_heads) * D;
      w[i][0].load(src + 8 * g0);
      w[i][1].load(src + 8 * g1);
    } else {
#pragma unroll
      for (int e = 0; e < Eight<T>::kVecs; ++e) w[i][0].w[e] = w[i][1].w[e] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  int64_t at = -1;
  if (live) {
    at = __ldg(a.positions + t);
    live = at >= 0;
    if (live && a.position_offsets) at += __ldg(a.position_offsets + t);
    if (live && a.rotary_dim > 0 && (at < 0 || at >= a.max_position)) {
      if (first == 0 && j == 0) record_error(p.err, PA_DEVERR_POSITION);
      live = false;
    }
  }
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
  if (live && turns) {
    const float* row = a.cos_sin + at * a.rotary_dim + 8 * j;
    const uint4 v[4] = {ldg_nc_v4(row), ldg_nc_v4(row + 4), ldg_nc_v4(row + a.rotary_dim / 2),
                        ldg_nc_v4(row + a.rotary_dim / 2 + 4)};
    ElemTraits<float>::unpack(v[0], c);
    ElemTraits<float>::unpack(v[1], c + 4);
    ElemTraits<float>::unpack(v[2], s);
    ElemTraits<float>::unpack(v[3], s + 4);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = first + i * p.groups;
    const bool is_key = h >= a.num_heads;
    float x[16];
    w[i][0].unpack(x);
    w[i][1].unpack(x + 8);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!live || h >= heads) continue;
    const float inv = __frsqrt_rn(fmaf(sum, 1.f / D, a.eps));
    const T* weight = static_cast<const T*>(is_key ? a.key_weight : a.query_weight);
    if (weight) {
      float y[16];
      Eight<T> w0, w1;
      w0.load(weight + 8 * g0);
      w1.load(weight + 8 * g1);
      w0.unpack(y);
      w1.unpack(y + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * y[e];
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= inv;
    }
    if (turns) {
      auto turn = [&](float& u, float& v, int e) {
        const float nu = u * c[e] - v * s[e];
        v = v * c[e] + u * s[e];
        u = nu;
      };
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn(x[2 * e], x[2 * e + 1], e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn(x[e], x[e + 8], e);
      }
    }
    T* dst = is_key ? static_cast<T*>(a.key_out) + t * a.key_out_stride + (h - a.num_heads) * D
                    : static_cast<T*>(a.query_out) + t * a.query_out_stride + h * D;
    Eight<T>::store(dst + 8 * g0, x);
    Eight<T>::store(dst + 8 * g1, x + 8);
  }
}

template <typename T, int D, int N>
cudaError_t launch_heads(RopeParams p, cudaStream_t stream) {
  constexpr int kRows = kRopeThreads / (D / 16);  // of a CTA
  p.groups = (p.a.num_heads + p.a.num_kv_heads + N - 1) / N;
  const int64_t grid = ((int64_t)p.a.num_tokens * p.groups + kRows - 1) / kRows;
  void* args[] = {&p};
  return launch_overlapped((const void*)norm_rope_kernel<T, D, N>, dim3((unsigned)grid),
                           dim3(kRopeThreads), 0, stream, args);
}

template <typename T, int D>
cudaError_t launch(const pa_norm_rope_args& args, int num_sms, unsigned int* err,
                   cudaStream_t stream) {
  RopeParams p;
  p.a = args;
  p.err = err;
  constexpr int kMost = sizeof(T) == 2 ? 4 : 2;
  // Several heads a thread where there are more rows than the GPU's lanes hold at once.
  const int64_t rows = (int64_t)args.num_tokens * (args.num_heads + args.num_kv_heads);
  if (rows * (D / 16) <= 2048ll * num_sms) return launch_heads<T, D, 1>(p, stream);
  return launch_heads<T, D, kMost>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const pa_norm_rope_args& args, int num_sms, unsigned int* err,
                             cudaStream_t stream) {
  const bool half = args.dtype == PA_BF16;
  switch (args.head_size) {
    case 64:
      return half ? launch<__nv_bfloat16, 64>(args, num_sms, err, stream)
                  : launch<float, 64>(args, num_sms, err, stream);
    case 128:
      return half ? launch<__nv_bfloat16, 128>(args, num_sms, err, stream)
                  : launch<float, 128>(args, num_sms, err, stream);
    default:
      return half ? launch<__nv_bfloat16, 256>(args, num_sms, err, stream)
                  : launch<float, 256>(args, num_sms, err, stream);
  }
}

}  // namespace pa
