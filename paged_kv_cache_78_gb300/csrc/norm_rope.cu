// Norms of queries and keys for each head, and the rotation by position, in one pass for
// sm_103a (pa_norm_rope).
//
// Every element is read once and written once: memory, and for bf16 the instructions (about 12
// an element).  A head's row goes over D / 16 lanes, 16 elements each, which are eight pairs: the lane's
// two groups of eight neighbours are the pairs' first and second elements (halves), or the
// pairs lie inside the groups (neighbours).  Either way the lane's cosines and sines are eight in a
// row of the table, and no element leaves its lane.  A token's heads are shared out over lanes that
// go through them with the same cosines; products go two to an instruction.
//
// Measured (graph replays in a row, data larger than L2): 16381 tokens, 32 + 8 heads of 128, bf16
// 60.4 us (5.7 TB/s, 84% of the copy rate), fp32 100 us (6.8 TB/s, 100%); heads of 256 55 us (8192 tokens),
// 128 tokens 2.3 us, 64 of 14 + 2 heads of 64 1.7 us.  (With the next heads on their way to shared memory,
// two stages a thread: the same, fp32 half as long again.)
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

// CTAs of four warps leave the SM's last wave the least to wait for (512 tokens of 40 heads 3.7 us; 30%
// longer with eight warps, 24% with two).
constexpr int kRopeThreads = 128;

struct RopeParams {
  pa_norm_rope_args a;
  unsigned int* err;
  int groups;  // rows of lanes that share a token's heads
};

__device__ __forceinline__ Two negative(Two a) { return Two{a.v ^ 0x8000000080000000ull}; }

// Eight neighbours as four pairs of fp32, and back.
template <typename T>
struct Eight {
  static constexpr int kVecs = sizeof(T) / 2;
  uint4 w[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void unpack(Two* x) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) ElemTraits<T>::unpack(w[i], f + i * ElemTraits<T>::kPerChunk);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = two(f[2 * i], f[2 * i + 1]);
  }
  static __device__ __forceinline__ void store(T* p, const Two* x) {
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = parts(x[i]);
    if constexpr (sizeof(T) == 2) {
      stg_v4(p, make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                           pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y)));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        stg_v4(p + 4 * i, make_uint4(__float_as_uint(f[2 * i].x), __float_as_uint(f[2 * i].y),
                                     __float_as_uint(f[2 * i + 1].x), __float_as_uint(f[2 * i + 1].y)));
    }
  }
};

// Where a row of lanes stands: a token, and the first of its heads that are the row's (every
// p.groups-th is).
struct Place {
  int64_t t;
  int first;
};
__device__ __forceinline__ Place place_of(const RopeParams& p, unsigned unit) {
  const unsigned token = unit / (unsigned)p.groups;
  return Place{(int64_t)token, (int)(unit - token * p.groups)};
}
template <typename T>
__device__ __forceinline__ const T* row_in(const pa_norm_rope_args& a, int64_t t, int h) {
  return h < a.num_heads ? static_cast<const T*>(a.query) + t * a.query_stride + h * a.head_size
                         : static_cast<const T*>(a.key) + t * a.key_stride +
                               (h - a.num_heads) * a.head_size;
}

// What a lane knows of its part of a row.
struct Lane {
  int j, g0, g1;  // its number, and its two groups of eight
  bool turns;
};
__device__ __forceinline__ Lane lane_of(const pa_norm_rope_args& a, int j) {
  const int half = a.rotary_dim / 16;  // lanes that rotate
  Lane l;
  l.j = j;
  l.turns = j < half;
  l.g0 = a.interleaved || !l.turns ? 2 * j : j;
  l.g1 = a.interleaved || !l.turns ? 2 * j + 1 : j + half;
  return l;
}

// The token's position; false for padding and for positions past the table, which `report`
// records.
__device__ __forceinline__ bool position_of(const RopeParams& p, int64_t t, int64_t* at, bool report) {
  const pa_norm_rope_args& a = p.a;
  *at = __ldg(a.positions + t);
  if (*at < 0) return false;
  if (a.position_offsets) *at += __ldg(a.position_offsets + t);
  if (a.rotary_dim > 0 && (*at < 0 || *at >= a.max_position)) {
    if (report) record_error(p.err, PA_DEVERR_POSITION);
    return false;
  }
  return true;
}

// Cosines and sines of the lane's eight pairs, in a row of the table.
__device__ __forceinline__ void angles_of(const pa_norm_rope_args& a, const Lane& l, int64_t at,
                                          bool live, Two* c, Two* s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = two(1.f, 1.f), s[e] = two(0.f, 0.f);
  if (live && l.turns) {
    const float* row = a.cos_sin + at * a.rotary_dim + 8 * l.j;
    Eight<float> v;
    v.w[0] = ldg_nc_v4(row), v.w[1] = ldg_nc_v4(row + 4);
    v.unpack(c);
    v.w[0] = ldg_nc_v4(row + a.rotary_dim / 2), v.w[1] = ldg_nc_v4(row + a.rotary_dim / 2 + 4);
    v.unpack(s);
  }
}

// One head of a token, in the lanes of a row.  All of the warp's lanes come along.
template <typename T, int D>
__device__ __forceinline__ void turn_head(const pa_norm_rope_args& a, const Lane& l, int64_t t, int h,
                                          bool on, const Eight<T>& w0, const Eight<T>& w1,
                                          const Two* c, const Two* s) {
  Two x[8];
  w0.unpack(x);
  w1.unpack(x + 4);
  Two squares = x[0] * x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) squares = fma2(x[e], x[e], squares);
  float sum = parts(squares).x + parts(squares).y;
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (!on) return;
  const bool is_key = h >= a.num_heads;
  const float inv = rsqrtf(fmaf(sum, 1.f / D, a.eps));
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = x[e] * two(inv, inv);
  const T* weight = static_cast<const T*>(is_key ? a.key_weight : a.query_weight);
  if (weight) {
    Two y[4];
    Eight<T> g;
    g.load(weight + 8 * l.g0);
    g.unpack(y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = x[e] * y[e];
    g.load(weight + 8 * l.g1);
    g.unpack(y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e + 4] = x[e + 4] * y[e];
  }
  if (!a.interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const Two u = x[e], v = x[e + 4];
      x[e] = fma2(u, c[e], v * negative(s[e]));
      x[e + 4] = fma2(u, s[e], v * c[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 uv = parts(x[e]);
      const float ce = e % 2 ? parts(c[e / 2]).y : parts(c[e / 2]).x;
      const float se = e % 2 ? parts(s[e / 2]).y : parts(s[e / 2]).x;
      x[e] = two(uv.x * ce - uv.y * se, uv.y * ce + uv.x * se);
    }
  }
  T* dst = is_key ? static_cast<T*>(a.key_out) + t * a.key_out_stride + (h - a.num_heads) * D
                  : static_cast<T*>(a.query_out) + t * a.query_out_stride + h * D;
  Eight<T>::store(dst + 8 * l.g0, x);
  Eight<T>::store(dst + 8 * l.g1, x + 4);
}

// A row of lanes has N heads of a token, all of which it asks for at once and before it knows
// the position.
template <typename T, int D, int N>
__global__ void __launch_bounds__(kRopeThreads, 8)
    norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;
  const pa_norm_rope_args& a = p.a;
  const Place at = place_of(p, blockIdx.x * (kRopeThreads / kLanes) + threadIdx.x / kLanes);
  const Lane l = lane_of(a, threadIdx.x % kLanes);
  const int heads = a.num_heads + a.num_kv_heads;
  grid_dependents_launch();
  grid_dependency_wait();
  bool live = at.t < a.num_tokens;  // lanes of other tokens share the warp
  Eight<T> w[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = at.first + i * p.groups;
    if (live && h < heads) {
      const T* src = row_in<T>(a, at.t, h);
      w[i][0].load(src + 8 * l.g0);
      w[i][1].load(src + 8 * l.g1);
    } else {
      w[i][0].clear();
      w[i][1].clear();
    }
  }
  int64_t pos = 0;
  live = live && position_of(p, at.t, &pos, at.first == 0 && l.j == 0);
  Two c[4], s[4];
  angles_of(a, l, pos, live, c, s);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = at.first + i * p.groups;
    turn_head<T, D>(a, l, at.t, h, live && h < heads, w[i][0], w[i][1], c, s);
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
  // 96 bytes of a thread (fp32 128) on their way at once where there are more rows than the GPU's
  // threads hold: 16381 tokens of 40 heads of 128, bf16, take 1% longer with two heads a thread than with
  // three, 27% with one (four leave registers for fewer warps: 0.3%, heads of 256 2%); fp32 8% longer
  // with one than with two.
  const int64_t rows = (int64_t)args.num_tokens * (args.num_heads + args.num_kv_heads);
  if (rows * (D / 16) <= 2048ll * num_sms) return launch_heads<T, D, 1>(p, stream);
  return launch_heads<T, D, sizeof(T) == 2 ? 3 : 2>(p, stream);
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
