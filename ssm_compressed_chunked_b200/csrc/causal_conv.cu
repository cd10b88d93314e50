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
// 4 channels and walks a run of tokens with the last K-1 inputs in registers, so
// each input is read once but for the K-1 rows ahead of the run.  A warp has 128
// neighbouring channels, a block four warps of one run.  Rows come through a ring of
// the thread's own in shared memory, 16 rows deep (cp.async, no barrier): held in
// registers, the same rows in flight cost the blocks that hide the latency.
// 32768 x 2048, K 4, bf16: 50 us in a graph of such calls, 52 with other work between
// them, 5.1-5.4 TB/s (80-83% of the copy rate); f32 88 us, 6.1 TB/s (94%).  bf16 rows
// loaded into registers four or eight at a time 62, sixteen 74, one batch ahead 60-70.
// SiLU takes two operations an element on the multi-function unit (65% busy in bf16).
// A width that leaves most of the last block's warps without channels pays for them:
// 32768 x 640 bf16 25 us, x 512 18.
//
// Ownership.  The run that holds a sequence's first token (or an empty sequence's
// place) also computes that sequence's first K-1 tokens when they pass the run's
// end, and writes its window: the only thread that reads a carried window is then
// the thread that replaces it, so no order between blocks is needed.
#include "launch.h"
#include "ssm_block.cuh"

namespace attamba {

namespace {
constexpr int kConvWarps = 4;       // neighbouring groups of 32 channel vectors
constexpr int kStepWarps = 4;       // batch rows a block of the step
constexpr int kBatch = 4, kDepth = 4;   // rows copied together, batches in a thread's ring
constexpr int kV = 4;               // channels per thread

// kV channels of a row, as two pairs in fp32
static_assert(kV == 4, "two pairs");
template <typename T> struct Pack;
template <> struct Pack<float> {
  using raw = float4;
  static __device__ __forceinline__ raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void unpack(const raw& r, float2 (&v)[2]) {
    v[0] = make_float2(r.x, r.y);
    v[1] = make_float2(r.z, r.w);
  }
  static __device__ __forceinline__ raw pack(const float2 (&v)[2]) { return make_float4(v[0].x, v[0].y, v[1].x, v[1].y); }
};
template <> struct Pack<__nv_bfloat16> {
  using raw = uint2;
  static __device__ __forceinline__ raw zero() { return make_uint2(0, 0); }
  static __device__ __forceinline__ void unpack(const raw& r, float2 (&v)[2]) {
    v[0] = make_float2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
    v[1] = make_float2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
  }
  static __device__ __forceinline__ raw pack(const float2 (&v)[2]) {   // exact for values that came from unpack
    return make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
  }
};

// The taps and bias of a thread's channels, in the arithmetic's two-wide form.
template <typename T, int K> struct Taps {
  using raw = typename Pack<T>::raw;
  float2 w[K][2];
  float2 bias[2];
  __device__ __forceinline__ void load(const ConvArgs& p, int c0) {
    float f[kV * K];   // [channel][tap], as in memory
    const float4* src = reinterpret_cast<const float4*>(p.w + (size_t)c0 * K);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float4 v = __ldg(src + i);
      f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k][0] = make_float2(f[k], f[K + k]);
      w[k][1] = make_float2(f[2 * K + k], f[3 * K + k]);
    }
    const float4 b = p.bias ? __ldg(reinterpret_cast<const float4*>(p.bias + c0)) : make_float4(0.f, 0.f, 0.f, 0.f);
    bias[0] = make_float2(b.x, b.y);
    bias[1] = make_float2(b.z, b.w);
  }
  // win: inputs t-(K-1) .. t-1, xr: input t; returns y_t and moves the window on by one
  template <bool SILU>
  __device__ __forceinline__ raw step(float2 (&win)[K - 1][2], const raw& xr) const {
    float2 acc[2], x[2];
    Pack<T>::unpack(xr, x);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      acc[i] = bias[i];
#pragma unroll
      for (int k = 0; k < K; ++k) acc[i] = fma2(w[k][i], k < K - 1 ? win[k][i] : x[i], acc[i]);
      if (SILU) acc[i] = silu2(acc[i]);
#pragma unroll
      for (int k = 0; k + 1 < K - 1; ++k) win[k][i] = win[k + 1][i];
      win[K - 2][i] = x[i];
    }
    return Pack<T>::pack(acc);
  }
};

// block: one run of `run` tokens of up to kConvWarps neighbouring groups of 32 channel vectors, a warp each
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(32 * kConvWarps) causal_conv_kernel(ConvArgs p, int run) {
  using raw = typename Pack<T>::raw;
  __shared__ __align__(16) raw ring[kDepth][kBatch][32 * kConvWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int width = blockDim.x * kV;                       // channels a block
  const int groups = (p.D + width - 1) / width;
  const int group = blockIdx.x % groups;
  const int64_t t0 = (int64_t)(blockIdx.x / groups) * run;
  if (blockIdx.x == 0 && warp == 0) check_sequences_warp(p.cu, p.S, p.T, lane, p.status);
  const bool last_run = t0 + run >= p.T;
  const int total = max(0, (int)min((int64_t)p.cu[p.S], p.T));
  const int t1 = (int)min(t0 + run, (int64_t)total);
  const int c0 = group * width + (int)threadIdx.x * kV;
  const bool active = c0 < p.D;
  Taps<T, K> taps;
  if (active) taps.load(p, c0);
  const T* __restrict__ x = static_cast<const T*>(p.x) + c0;
  T* __restrict__ y = static_cast<T*>(p.y) + c0;
  T* st = static_cast<T*>(p.state) + c0;
  const raw zero = Pack<T>::zero();
  auto row = [&](int64_t t) { return __ldg(reinterpret_cast<const raw*>(x + t * p.ldx)); };

  float2 win[K - 1][2];
  // Tokens [a, b) of the sequence whose window is in win.  Batch g of kBatch rows is copied to slot g % kDepth
  // of the thread's own ring, kDepth - 1 batches ahead of the arithmetic; a group of copies per batch, empty
  // ones too, so that the wait counts batches.
  auto walk = [&](int a, int b) {
    if (!in_bounds(a >= 0 && b <= total && total <= p.T, p.status)) return;
    const T* src = x + (int64_t)a * p.ldx;
    auto fetch = [&](int g) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (a + g * kBatch + j < b) copy_async<sizeof(raw)>(&ring[g % kDepth][j][threadIdx.x], src + (int64_t)j * p.ldx);
      }
      src += (int64_t)kBatch * p.ldx;
      copies_commit();
    };
#pragma unroll
    for (int g = 0; g < kDepth - 1; ++g) fetch(g);
    T* dst = y + (int64_t)a * p.ldy;
    for (int t = a, g = 0; t < b; t += kBatch, ++g) {
      copies_wait<kDepth - 2>();
      fetch(g + kDepth - 1);
      const raw* r = &ring[g % kDepth][0][threadIdx.x];
      if (t + kBatch <= b) {   // whole: the window moves by renaming registers and no row is tested
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          *reinterpret_cast<raw*>(dst + (int64_t)j * p.ldy) = taps.template step<SILU>(win, r[j * 32 * kConvWarps]);
      } else {
#pragma unroll
        for (int j = 0; j < kBatch - 1; ++j)
          if (t + j < b)
            *reinterpret_cast<raw*>(dst + (int64_t)j * p.ldy) = taps.template step<SILU>(win, r[j * 32 * kConvWarps]);
      }
      dst += (int64_t)kBatch * p.ldy;
    }
    copies_wait<0>();
  };

  // the first sequence that starts at t0 or later; the one before it may reach into this run, whose share of it
  // begins behind its first K-1 tokens (they belong to the run that it starts in)
  const int s0 = count_below_warp(p.cu, p.S, (int)t0, lane);
  int64_t from = 0;
  bool reaches = false;
  if (s0 > 0) {
    from = max(t0, (int64_t)max(0, p.cu[s0 - 1]) + K - 1);
    reaches = from < min(p.cu[s0], t1);
  }
  for (int s = reaches ? s0 - 1 : s0; s < p.S; ++s) {
    int a, b, end = 0, slot = -1;
    if (s < s0) {
      a = (int)from;
      b = min(p.cu[s0], t1);
      if (active) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) Pack<T>::unpack(row(a - (K - 1) + k), win[k]);
      }
    } else {
      const int cs = p.cu[s];
      if (cs >= t0 + run && !last_run) break;
      a = min(max(cs, (int)min(t0, (int64_t)total)), total);   // clamps act on a malformed cu only
      end = min(max(p.cu[s + 1], a), total);
      b = min(end, max(t1, a + K - 1));
      if (p.state) slot = state_slot_warp(p.slots, s, p.n_slots, lane, p.status);
      const bool kept = active && slot >= 0 && p.cont && p.cont[s] != 0;
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
        Pack<T>::unpack(kept ? *reinterpret_cast<const raw*>(st + ((size_t)slot * (K - 1) + k) * p.D) : zero, win[k]);
    }
    if (!active) continue;
    walk(a, b);
    if (slot >= 0) {
      // the sequence's last K-1 inputs: in win when the walk reached its end, else K-1 rows that lie in it
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
        *reinterpret_cast<raw*>(st + ((size_t)slot * (K - 1) + k) * p.D) =
            b < end && in_bounds(end - (K - 1) >= 0 && end <= total, p.status) ? row(end - (K - 1) + k) : Pack<T>::pack(win[k]);
    }
  }
}

// grid: x = groups of kStepWarps batch rows, y = groups of 32 channel vectors
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(32 * kStepWarps) conv_step_kernel(ConvArgs p) {
  using raw = typename Pack<T>::raw;
  __shared__ SlotTable table;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = blockIdx.x * kStepWarps, b = first + warp;
  // every load goes out before the slot is known to be good: one in range is safe to read
  const int slot = b < p.T ? (p.slots ? __ldg(p.slots + b) : b) : -1;
  const int c0 = (blockIdx.y * 32 + lane) * kV;
  const bool active = c0 < p.D && slot != -1;
  T* st = static_cast<T*>(p.state) + (size_t)(slot >= 0 && slot < p.n_slots ? slot : 0) * (K - 1) * p.D + c0;
  Taps<T, K> taps;
  float2 win[K - 1][2];
  raw x;
  if (active) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) Pack<T>::unpack(*reinterpret_cast<const raw*>(st + (size_t)k * p.D), win[k]);
    x = __ldg(reinterpret_cast<const raw*>(static_cast<const T*>(p.x) + (int64_t)b * p.ldx + c0));
    taps.load(p, c0);
  }
  const int good = state_slots_block(p.slots, first, 1, min((int)p.T, first + kStepWarps), p.n_slots, table, p.status);
  if (__shfl_sync(0xffffffffu, good, warp) < 0 || !active) return;
  *reinterpret_cast<raw*>(static_cast<T*>(p.y) + (int64_t)b * p.ldy + c0) = taps.template step<SILU>(win, x);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) *reinterpret_cast<raw*>(st + (size_t)k * p.D) = Pack<T>::pack(win[k]);
}

template <typename T, int K>
cudaError_t conv_prompts(const ConvArgs& a, cudaStream_t s) {
  const int warps = min((a.D + 32 * kV - 1) / (32 * kV), kConvWarps);
  const int64_t groups = (a.D + 32 * kV * warps - 1) / (32 * kV * warps);
  // Long runs read less ahead of themselves and start fewer blocks; short ones fill the SMs when there are few tokens
  // (B200, us at runs of 16 / 32 / 64: 32768 x 2048 bf16 62.4 / 51.8 / 48.5, 2048 x 2048 bf16 5.9 / 6.1 / 7.7).
  int run = 64;
  while (run > 8 && groups * ((a.T + run - 1) / run) < (run > 16 ? 1024 : 256)) run /= 2;
  const int64_t blocks = groups * ((a.T + run - 1) / run);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return a.act == ATTAMBA_ACT_SILU
             ? launch_dependent(causal_conv_kernel<T, K, true>, dim3((unsigned)blocks), 32 * warps, s, a, run)
             : launch_dependent(causal_conv_kernel<T, K, false>, dim3((unsigned)blocks), 32 * warps, s, a, run);
}

template <typename T, int K>
cudaError_t conv_step(const ConvArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.T + kStepWarps - 1) / kStepWarps), (a.D + 32 * kV - 1) / (32 * kV));
  return a.act == ATTAMBA_ACT_SILU ? launch_dependent(conv_step_kernel<T, K, true>, grid, 32 * kStepWarps, s, a)
                                   : launch_dependent(conv_step_kernel<T, K, false>, grid, 32 * kStepWarps, s, a);
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
