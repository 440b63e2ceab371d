// Rotary positions (misa_rope in misa.h).
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace misa {

namespace {

struct RopeArgs {
  Rope s;
  int32_t n, row;  // row: heads * d
  const void* x;
  const int32_t* pos;
  const double* freq;
  void* out;
  float* out_scale;
};

// amplitude * (cos, sin) of pos * freq.  The product's whole turns, and what its
// rounding lost, are taken care of in 64 bits; what is left is below half a turn.
__device__ __forceinline__ float2 turn(int32_t pos, double freq, float amplitude) {
  const double f = freq * 0.15915494309189533577;  // 1 / (2 pi)
  const double p = pos, t = p * f;
  const float r = static_cast<float>((t - rint(t)) + fma(p, f, -t));
  float c, s;
  sincospif(2.f * r, &s, &c);
  return make_float2(amplitude * c, amplitude * s);
}

__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float y = a * cs.x - b * cs.y;
  b = a * cs.y + b * cs.x;
  a = y;
}

// Eight values of X at element `at` (a multiple of 8) of p.
template <int X>
__device__ __forceinline__ void load8(const void* p, int64_t at, float* y) {
  if constexpr (X == kF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 u = q[0], v = q[1];
    y[0] = u.x; y[1] = u.y; y[2] = u.z; y[3] = u.w;
    y[4] = v.x; y[5] = v.y; y[6] = v.z; y[7] = v.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = __uint_as_float(w[j] << 16);
      y[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

template <int OUT>
__device__ __forceinline__ void store8(void* p, int64_t at, const float* y) {
  if constexpr (OUT == kF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    q[0] = make_float4(y[0], y[1], y[2], y[3]);
    q[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else if constexpr (OUT == kBF16) {
    typedef __attribute__((ext_vector_type(8))) __bf16 B8;
    B8 b;
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = static_cast<__bf16>(y[j]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = __builtin_bit_cast(uint4, b);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + at) =
        make_uint2(e4m3_pack4(y[0], y[1], y[2], y[3], 1.f), e4m3_pack4(y[4], y[5], y[6], y[7], 1.f));
  }
}

constexpr int kTurns = 2048;  // (cos, sin) pairs in LDS: of all of a workgroup's tokens

// TPR threads a token, 256 / TPR tokens a workgroup.  An item is 16 elements of a
// head: eight pairs of the rotated part (in the half layout two runs of eight,
// rot / 2 apart), or 16 neighbours of the rest.  The heads of a token share its
// angles: they are computed once into LDS while the values' loads are under way,
// and the values stay in registers until the token's largest magnitude is known.
//
// Bound by memory traffic: 8192 tokens of 64 heads of 128, bf16 to e4m3 (201 MB) 41.6
// us, 4.8 TB/s, to bf16 50.9 us, 5.3 TB/s; 32 tokens of 72 heads 4.2 us, a launch, the
// angles and the loads.
template <int X, int OUT, int TPR, int NI>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  constexpr int TOKENS = 256 / TPR;
  __shared__ __attribute__((aligned(16))) float2 turns[kTurns];
  __shared__ float tops[4];
  const Rope& s = a.s;
  const int sub = threadIdx.x % TPR, tok = threadIdx.x / TPR;
  const int32_t t0 = blockIdx.x * TOKENS, t = t0 + tok;
  const bool live = t < a.n;
  const int per_head = s.d / 16, items = s.heads * per_head, half = s.rot / 2;
  const int first = s.first / 16, rotated = s.rot / 16;
  const int64_t from = static_cast<int64_t>(t) * s.x_stride, to = static_cast<int64_t>(t) * s.out_stride;
  const bool pass = OUT == kFP8 || a.x != a.out;  // the rest is there already

  float y[NI][16];
  int32_t at[NI], gap[NI], angle[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int item = i * TPR + sub;
    const int head = item / per_head, c = item - head * per_head - first;
    const bool turned = c >= 0 && c < rotated;
    angle[i] = turned ? 8 * c : -1;
    at[i] = head * s.d + s.first + (turned && s.pairs == 0 ? 8 : 16) * c;
    gap[i] = turned && s.pairs == 0 ? half : 8;
    if (!live || item >= items || (!turned && !pass)) {
      at[i] = -1;
#pragma unroll
      for (int j = 0; j < 16; ++j) y[i][j] = 0.f;
    } else {
      load8<X>(a.x, from + at[i], y[i]);
      load8<X>(a.x, from + at[i] + gap[i], y[i] + 8);
    }
  }
  for (int i = threadIdx.x; i < TOKENS * half; i += 256) {
    const int32_t tt = t0 + i / half;
    if (tt < a.n) turns[i] = turn(a.pos[tt], a.freq[i % half], s.amplitude);
  }
  __syncthreads();
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (at[i] >= 0 && angle[i] >= 0) {
      float2 cs[8];
      const float4* src = reinterpret_cast<const float4*>(turns + tok * half + angle[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = src[j];
        cs[2 * j] = make_float2(v.x, v.y);
        cs[2 * j + 1] = make_float2(v.z, v.w);
      }
      if (s.pairs == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) rotate(y[i][j], y[i][8 + j], cs[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) rotate(y[i][2 * j], y[i][2 * j + 1], cs[j]);
      }
    }
    if constexpr (OUT == kFP8) {
#pragma unroll
      for (int j = 0; j < 16; ++j) top = amax_step(top, y[i][j]);
    }
  }
  if constexpr (OUT == kFP8) {
    top = lanes_reduce<(TPR < kWave ? TPR : kWave), true>(top);
    if constexpr (TPR > kWave) {
      if (lane_id() == 0) tops[threadIdx.x / kWave] = top;
      __syncthreads();
      top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    }
    float scale, mult;
    e4m3_scale(top, scale, mult);
    if (sub == 0 && live) a.out_scale[t] = scale;
    const Quotient by_scale(scale);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) y[i][j] = by_scale.of(y[i][j]);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (at[i] < 0) continue;
    store8<OUT>(a.out, to + at[i], y[i]);
    store8<OUT>(a.out, to + at[i] + gap[i], y[i] + 8);
  }
}

// Sizes and strides off the runs of 16 (4096 tokens of 32 heads of 72, 36 of them
// turned: 21 us, 1.8 TB/s): a workgroup per token, a thread per pair or passing
// element, angles computed where they are needed; an 8-bit output goes through the
// values twice.  Bound by the angles, in 64 bits and anew for each head, and by loads
// and stores of single elements.
template <int X, int OUT>
__global__ __launch_bounds__(256) void rope_any_kernel(RopeArgs a) {
  __shared__ float tops[4];
  const Rope& s = a.s;
  const int32_t t = blockIdx.x;
  const int64_t from = static_cast<int64_t>(t) * s.x_stride, to = static_cast<int64_t>(t) * s.out_stride;
  const int half = s.rot / 2, per_head = s.d - half;  // pairs, then the rest
  const int32_t pos = a.pos[t];
  float scale = 1.f, mult = 1.f, top = 0.f;
  for (int round = OUT == kFP8 ? 0 : 1; round < 2; ++round) {
    const Quotient by_scale(scale);  // known from the first round
    for (int i = threadIdx.x; i < s.heads * per_head; i += 256) {
      const int head = i / per_head, e = i - head * per_head;
      int p = s.first + e, q = -1;
      if (e < half) {
        p = s.first + (s.pairs == 0 ? e : 2 * e);
        q = p + (s.pairs == 0 ? half : 1);
      } else {
        p = e - half < s.first ? e - half : e + half;
      }
      p += head * s.d;
      q += q < 0 ? 0 : head * s.d;
      float x0 = load_elem<X>(a.x, from + p), x1 = 0.f;
      if (q >= 0) {
        x1 = load_elem<X>(a.x, from + q);
        rotate(x0, x1, turn(pos, a.freq[e], s.amplitude));
      }
      if (round == 0) {
        top = amax_step(amax_step(top, x0), x1);
        continue;
      }
      if constexpr (OUT == kF32) {
        static_cast<float*>(a.out)[to + p] = x0;
        if (q >= 0) static_cast<float*>(a.out)[to + q] = x1;
      } else if constexpr (OUT == kBF16) {
        static_cast<__bf16*>(a.out)[to + p] = static_cast<__bf16>(x0);
        if (q >= 0) static_cast<__bf16*>(a.out)[to + q] = static_cast<__bf16>(x1);
      } else {
        const uint32_t code = e4m3_pack4(by_scale.of(x0), by_scale.of(x1), 0.f, 0.f, 1.f);
        static_cast<uint8_t*>(a.out)[to + p] = static_cast<uint8_t>(code);
        if (q >= 0) static_cast<uint8_t*>(a.out)[to + q] = static_cast<uint8_t>(code >> 8);
      }
    }
    if (round == 0) {
      top = lanes_reduce<kWave, true>(top);
      if (lane_id() == 0) tops[threadIdx.x / kWave] = top;
      __syncthreads();
      e4m3_scale(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])), scale, mult);
      if (threadIdx.x == 0) a.out_scale[t] = scale;
    }
  }
}

// As few threads a token as hold its items one each, up to 256, so that a workgroup's
// tokens fill it: 131072 tokens of one head of 128 18.8 us with 16, 37.9 with 64; 32768 of 8
// heads 27.8 with 64, 37.2 with 256 and 30.4 with 16 of four items each; 8192 of 32 heads
// 28.5 with 256, 30.8 with 64 of four.  Runs of 16 take 51.0 us for 8192 tokens of 64 heads, 114.6 in
// single elements; 4096 of 32 heads of 80 10.4 and 22.9.
template <int X, int OUT>
hipError_t launch_types(const RopeArgs& a, hipStream_t st) {
  const Rope& s = a.s;
  const bool runs = s.d % 16 == 0 && s.first % 16 == 0 && s.rot % 16 == 0 && s.x_stride % 8 == 0 && s.out_stride % 8 == 0;
  const int items = a.row / 16;
  if (!runs) {
    rope_any_kernel<X, OUT><<<a.n, 256, 0, st>>>(a);
  } else if (items <= 16) {
    rope_kernel<X, OUT, 16, 1><<<(a.n + 15) / 16, 256, 0, st>>>(a);
  } else if (items <= 64) {
    rope_kernel<X, OUT, 64, 1><<<(a.n + 3) / 4, 256, 0, st>>>(a);
  } else if (items <= 256) {
    rope_kernel<X, OUT, 256, 1><<<a.n, 256, 0, st>>>(a);
  } else if (items <= 512) {
    rope_kernel<X, OUT, 256, 2><<<a.n, 256, 0, st>>>(a);
  } else if (items <= 1024) {
    rope_kernel<X, OUT, 256, 4><<<a.n, 256, 0, st>>>(a);
  } else {
    rope_kernel<X, OUT, 256, 8><<<a.n, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

template <int X>
hipError_t launch_out(const RopeArgs& a, hipStream_t st) {
  switch (a.s.out_dtype) {
    case kF32: return launch_types<X, kF32>(a, st);
    case kBF16: return launch_types<X, kBF16>(a, st);
    default: return launch_types<X, kFP8>(a, st);
  }
}

}  // namespace

hipError_t launch_rope(const Rope& r, int32_t n, const void* x, const int32_t* pos,
                       const double* freq, void* out, float* out_scale, hipStream_t st) {
  const RopeArgs a{r, n, r.heads * r.d, x, pos, freq, out, out_scale};
  return r.x_dtype == kF32 ? launch_out<kF32>(a, st) : launch_out<kBF16>(a, st);
}

}  // namespace misa
