// Short causal depthwise convolution over packed prompts, and its single-token step.
//
// Method: pith.science review of Attamba, "Assumptions & free parameters" -- the
// SSM is Mamba's selective SSM, whose block passes the input through a short
// convolution first.  Per token t, channel d, K = 2, 3 or 4 taps:
//     y[t,d] = act(bias[d] + sum_{k<K} w[d,k] x[t-(K-1)+k, d]),
// positions ahead of the sequence's first token from its carried window (the last
// K-1 inputs of what came before) or zero.
//
// Mapping (B200).  Memory-bound: one read and one write of [T, D].  A thread owns
// 16 bytes of channels (8 bf16 or 4 f32) and walks a run of tokens with the last
// K-1 inputs in registers, so each input is read once but for the K-1 rows ahead
// of the run.  A warp is 32 neighbouring channel vectors of one run: its accesses
// are whole 512-byte lines of a row.
//
// Ownership.  The run that holds a sequence's first token (or an empty sequence's
// place) also computes that sequence's first K-1 tokens when they pass the run's
// end, and writes its window: the only thread that reads a carried window is then
// the thread that replaces it, so no order between blocks is needed.
#include "common.cuh"
#include "launch.h"

namespace attamba {

namespace {
constexpr int kConvThreads = 128;   // 4 warps, each with its own run of tokens
constexpr int kConvWarps = kConvThreads / 32;
constexpr int kAhead = 4;           // rows loaded together

// 16 bytes of channels as fp32
template <typename T> struct Pack;
template <> struct Pack<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <> struct Pack<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};

// The taps and bias of a thread's channels.
template <typename T, int K> struct Taps {
  static constexpr int V = Pack<T>::kN;
  float w[K][V];
  float bias[V];
  __device__ __forceinline__ void load(const ConvArgs& p, int c0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][i] = __ldg(p.w + (size_t)(c0 + i) * K + k);
      bias[i] = p.bias ? __ldg(p.bias + c0 + i) : 0.f;
    }
  }
  // win: inputs t-(K-1) .. t-1, x: input t; returns y_t and moves the window on by one
  __device__ __forceinline__ uint4 step(uint4 (&win)[K - 1], const uint4& x, int act) const {
    float acc[V], v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = bias[i];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Pack<T>::unpack(k < K - 1 ? win[k] : x, v);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(w[k][i], v[i], acc[i]);
    }
    if (act == ATTAMBA_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = silu_f(acc[i]);
    }
#pragma unroll
    for (int k = 0; k + 1 < K - 1; ++k) win[k] = win[k + 1];
    win[K - 2] = x;
    return Pack<T>::pack(acc);
  }
};

// block: kConvWarps runs of `run` tokens of one group of 32 channel vectors; a run's groups are neighbours
template <typename T, int K>
__global__ void __launch_bounds__(kConvThreads) causal_conv_kernel(ConvArgs p, int run) {
  constexpr int V = Pack<T>::kN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int groups = (p.D + 32 * V - 1) / (32 * V);
  const int group = blockIdx.x % groups;
  const int64_t t0 = ((int64_t)(blockIdx.x / groups) * kConvWarps + warp) * run;
  if (t0 >= p.T) return;
  if (group == 0 && t0 == 0) check_sequences_warp(p.cu, p.S, p.T, lane, p.status);
  const bool last_run = t0 + run >= p.T;
  const int total = max(0, (int)min((int64_t)p.cu[p.S], p.T));
  const int t1 = (int)min(t0 + run, (int64_t)total);
  const int c0 = (group * 32 + lane) * V;
  const bool active = c0 < p.D;
  Taps<T, K> taps;
  if (active) taps.load(p, c0);
  const T* __restrict__ x = static_cast<const T*>(p.x) + c0;
  T* __restrict__ y = static_cast<T*>(p.y) + c0;
  T* st = static_cast<T*>(p.state) + c0;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto row = [&](int64_t t) { return __ldg(reinterpret_cast<const uint4*>(x + t * p.ldx)); };
  auto put = [&](int64_t t, const uint4& v) { *reinterpret_cast<uint4*>(y + t * p.ldy) = v; };

  uint4 win[K - 1];
  // tokens [a, b) of the sequence whose window is in win
  auto walk = [&](int a, int b) {
    for (int t = a; t < b; t += kAhead) {
      uint4 r[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) r[j] = t + j < b ? row(t + j) : zero;
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (t + j < b) put(t + j, taps.step(win, r[j], p.act));
    }
  };

  // the first sequence that starts at t0 or later; the one before it may reach into this run
  int s = count_below_warp(p.cu, p.S, (int)t0, lane);
  if (s > 0 && active) {
    const int first = max(0, p.cu[s - 1]);
    const int64_t from = max(t0, (int64_t)first + K - 1);   // its first K-1 tokens belong to its first run
    const int b = min(p.cu[s], t1);
    if (from < b) {
      const int a = (int)from;
#pragma unroll
      for (int k = 0; k < K - 1; ++k) win[k] = row(a - (K - 1) + k);
      walk(a, b);
    }
  }
  for (; s < p.S; ++s) {
    const int cs = p.cu[s];
    if (cs >= t0 + run && !last_run) break;
    const int first = min(max(cs, (int)min(t0, (int64_t)total)), total);   // clamps act on a malformed cu only
    const int end = min(max(p.cu[s + 1], first), total);
    int slot = -1;
    if (p.state) slot = state_slot_warp(p.slots, s, p.n_slots, lane, p.status);
    if (!active) continue;
    uint4 old[K - 1];
    const bool kept = slot >= 0 && p.cont && p.cont[s] != 0;
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      old[k] = kept ? *reinterpret_cast<const uint4*>(st + ((size_t)slot * (K - 1) + k) * p.D) : zero;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) win[k] = old[k];
    walk(first, min(end, max(t1, first + K - 1)));
    if (slot >= 0) {
      // the last K-1 of (old window, inputs)
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {
        const int at = end - (K - 1) + k;
        uint4 v = zero;
        if (at >= first) {
          v = row(at);
        } else {
#pragma unroll
          for (int j = 0; j < K - 1; ++j)
            if (j == at - first + (K - 1)) v = old[j];
        }
        *reinterpret_cast<uint4*>(st + ((size_t)slot * (K - 1) + k) * p.D) = v;
      }
    }
  }
}

// grid: x = groups of kConvWarps batch rows, y = groups of 32 channel vectors
template <typename T, int K>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvArgs p) {
  constexpr int V = Pack<T>::kN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t b = (int64_t)blockIdx.x * kConvWarps + warp;
  if (b >= p.T) return;
  const int slot = state_slot_warp(p.slots, (int)b, p.n_slots, lane, p.status);
  const int c0 = (blockIdx.y * 32 + lane) * V;
  if (slot < 0 || c0 >= p.D) return;
  Taps<T, K> taps;
  taps.load(p, c0);
  T* st = static_cast<T*>(p.state) + (size_t)slot * (K - 1) * p.D + c0;
  uint4 win[K - 1];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) win[k] = *reinterpret_cast<const uint4*>(st + (size_t)k * p.D);
  const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + b * p.ldx + c0));
  *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + b * p.ldy + c0) = taps.step(win, x, p.act);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) *reinterpret_cast<uint4*>(st + (size_t)k * p.D) = win[k];
}

template <typename T, int K>
cudaError_t conv_prompts(const ConvArgs& a, cudaStream_t s) {
  const int run = 16;
  const int64_t groups = (a.D + 32 * Pack<T>::kN - 1) / (32 * Pack<T>::kN);
  const int64_t blocks = groups * ((a.T + run * kConvWarps - 1) / (run * kConvWarps));
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent(causal_conv_kernel<T, K>, dim3((unsigned)blocks), kConvThreads, s, a, run);
}

template <typename T, int K>
cudaError_t conv_step(const ConvArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.T + kConvWarps - 1) / kConvWarps), (a.D + 32 * Pack<T>::kN - 1) / (32 * Pack<T>::kN));
  return launch_dependent(conv_step_kernel<T, K>, grid, kConvThreads, s, a);
}
}  // namespace

cudaError_t launch_causal_conv(attamba_dtype_t dtype, int K, const ConvArgs& a, cudaStream_t s) {
  if (dtype == ATTAMBA_BF16)
    return K == 2 ? conv_prompts<__nv_bfloat16, 2>(a, s) : K == 3 ? conv_prompts<__nv_bfloat16, 3>(a, s)
                                                                   : conv_prompts<__nv_bfloat16, 4>(a, s);
  return K == 2 ? conv_prompts<float, 2>(a, s) : K == 3 ? conv_prompts<float, 3>(a, s) : conv_prompts<float, 4>(a, s);
}

cudaError_t launch_conv_step(attamba_dtype_t dtype, int K, const ConvArgs& a, cudaStream_t s) {
  if (dtype == ATTAMBA_BF16)
    return K == 2 ? conv_step<__nv_bfloat16, 2>(a, s) : K == 3 ? conv_step<__nv_bfloat16, 3>(a, s)
                                                                : conv_step<__nv_bfloat16, 4>(a, s);
  return K == 2 ? conv_step<float, 2>(a, s) : K == 3 ? conv_step<float, 3>(a, s) : conv_step<float, 4>(a, s);
}

}  // namespace attamba
