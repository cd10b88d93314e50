// The norms after a block and before the next one, with the block's gate, the
// residual scale and the residual sum, in one pass.
//
// Per row, with norm(v, w) = v rsqrt(mean(v^2) + eps) w:
//     v = y [act(gate)];  v = norm(v, w_post);  v = v [act(gate)];
//     r = res + alpha scale v;  h = norm(r, w_pre).
//
// Mapping (B200).  Memory-bound: y, gate and res read once, r and h written once.
// A row belongs to one block of 32 to 1024 threads (several rows a block while a warp
// holds a row); every thread has VPT vectors of 8 channels in fp32 registers
// from the first load to the last store, so the two means cost two reductions and
// no second read.  Sums of squares are fp32: a thread's share first, then the warp's
// tree, then the warps' partial sums.  16384 x 2048 bf16 with gate and fp32 residual:
// 71 us in a graph of such calls, 78 with other work between them, 6.0-6.6 TB/s (93-103%
// of the copy rate); f32 throughout, no gate: 82 us, 6.5 TB/s.
#include "launch.h"
#include "ssm_block.cuh"

namespace attamba {

namespace {
// 8 channels, as loaded and in fp32
template <typename T> struct Eight;
template <> struct Eight<float> {
  struct raw {
    float4 a, b;
  };
  static __device__ __forceinline__ raw get(const float* p) {
    return {*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4)};
  }
  static __device__ __forceinline__ void unpack(const raw& r, float (&v)[8]) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w; v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
  }
  static __device__ __forceinline__ void put(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Eight<__nv_bfloat16> {
  using raw = uint4;
  static __device__ __forceinline__ raw get(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void unpack(const raw& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};

__device__ __forceinline__ float act_f(int act, float g) {
  if (act == ATTAMBA_ACT_LINEAR) return g;
  const float s = sigmoid_f(g);
  return act == ATTAMBA_ACT_SILU ? g * s : s;
}

// Sum over the row's threads (32: the warp; more: the block, through `part`).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (TPR == 32) return v;
  __syncthreads();   // the partial sums of the sum before have been read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < TPR / 32; ++w) v += part[w];
  return v;
}

constexpr int kWarpRows = 4;   // rows a block while a warp holds a row

template <typename T, typename R, int TPR, int VPT>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kWarpRows : TPR) block_norm_kernel(NormArgs p) {
  __shared__ float part[TPR / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.M) return;   // whole warps only: a block of more threads has one row, below M
  const int id = threadIdx.x % TPR;
  const int D = p.D;
  // A thread with one vector loads all of its row first: the two sums would otherwise each put a memory latency ahead of the next
  // load (16384 x 2048, fp32 residual: 70.8 against 76.2 us).  With more vectors the registers that takes cost more
  // blocks than it gives (4096 x 8192: 65 against 56 us): there gate and residual are loaded where they are used, but
  // a bf16 residual waits in shared memory (8192 x 4096: 47.2 against 51.0 us, 4096 x 8192 52.8 against 56.3); an fp32
  // one takes twice the room and lost as much (4096 x 6000: 82.6 against 75.8).
  constexpr bool kFirst = VPT == 1, kAsync = VPT > 1 && sizeof(R) == 2 && TPR * VPT * 16 <= 32768;
  __shared__ __align__(16) typename Eight<R>::raw ahead[kAsync ? VPT : 1][kAsync ? TPR : 1];   // a thread's own pieces
  if (kAsync && p.res) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (id + k * TPR) * 8;
      if (c < D) copy_async<16>(&ahead[kAsync ? k : 0][kAsync ? id : 0], static_cast<const R*>(p.res) + row * p.ldr + c);
    }
    copies_commit();
  }
  float v[VPT][8];
  typename Eight<T>::raw g[VPT];
  typename Eight<R>::raw r[VPT];
  auto load_gate = [&](int k, int c) {
    g[k] = {};
    if (p.gate && c < D) g[k] = Eight<T>::get(static_cast<const T*>(p.gate) + row * p.ldg + c);
  };
  auto load_res = [&](int k, int c) {
    r[k] = {};
    if (p.res && c < D)
      r[k] = kAsync ? ahead[kAsync ? k : 0][kAsync ? id : 0] : Eight<R>::get(static_cast<const R*>(p.res) + row * p.ldr + c);
  };
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int c = (id + k * TPR) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
    if (p.y && c < D) Eight<T>::unpack(Eight<T>::get(static_cast<const T*>(p.y) + row * p.ldy + c), v[k]);
    if (kFirst) {
      load_gate(k, c);
      load_res(k, c);
    }
  }
  auto gate = [&]() {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float f[8];
      if (!kFirst) load_gate(k, (id + k * TPR) * 8);
      Eight<T>::unpack(g[k], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] *= act_f(p.act, f[i]);
    }
  };
  auto norm = [&](const float* w) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[k][i], v[k][i], ss);
    const float rs = rsqrtf(row_sum<TPR>(ss, part) / (float)D + p.eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (id + k * TPR) * 8;
      if (c < D) {
        float f[8];
        Eight<float>::unpack(Eight<float>::get(w + c), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= rs * f[i];
      }
    }
  };
  if (p.gate && p.gate_first) gate();
  if (p.w_post) norm(p.w_post);
  if (p.gate && !p.gate_first) gate();
  if (kAsync) copies_wait<0>();
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int c = (id + k * TPR) * 8;
    if (c >= D) continue;
    float f[8];
    if (p.scale) {
      Eight<float>::unpack(Eight<float>::get(p.scale + c), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] *= f[i];
    }
    if (!kFirst) load_res(k, c);
    Eight<R>::unpack(r[k], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = p.y ? fmaf(p.alpha, v[k][i], f[i]) : f[i];
    if (p.res_out) Eight<R>::put(static_cast<R*>(p.res_out) + row * p.ldro + c, v[k]);
  }
  if (p.h) {
    norm(p.w_pre);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (id + k * TPR) * 8;
      if (c < D) Eight<T>::put(static_cast<T*>(p.h) + row * p.ldh + c, v[k]);
    }
  }
}

template <typename T, typename R, int TPR, int VPT>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  const int64_t blocks = TPR == 32 ? (a.M + kWarpRows - 1) / kWarpRows : a.M;
  return launch_dependent(block_norm_kernel<T, R, TPR, VPT>, dim3((unsigned)blocks), TPR == 32 ? 32 * kWarpRows : TPR, s, a);
}

template <typename T, typename R>
cudaError_t launch_for(const NormArgs& a, cudaStream_t s) {
  // threads a row and vectors a thread, measured (B200, bf16 with a SiLU gate and both norms, 33.5M elements, GB/s of the
  // copy's 6470 with a bf16 / an fp32 residual): rows of 256 6500 / 6620, 512 6470 / 6640, 1024 6390 / 6640, 2048 6180 / 6600,
  // 4096 5230 / 5860, 8192 4860 / 5460, 16384 4140 / 4680, 32768 3550 / 4330; from 4096 on an SM holds too few rows to
  // overlap one's sums with another's loads
  const int vecs = a.D / 8;
  if (vecs <= 32) return launch<T, R, 32, 1>(a, s);
  if (vecs <= 64) return launch<T, R, 64, 1>(a, s);
  if (vecs <= 128) return launch<T, R, 128, 1>(a, s);
  if (vecs <= 256) return launch<T, R, 256, 1>(a, s);
  if (vecs <= 512) return launch<T, R, 256, 2>(a, s);
  if (vecs <= 1024) return launch<T, R, 512, 2>(a, s);
  if (vecs <= 2048) return launch<T, R, 512, 4>(a, s);
  return launch<T, R, 1024, 4>(a, s);
}
}  // namespace

cudaError_t launch_block_norm(attamba_dtype_t dtype, attamba_dtype_t res_dtype, const NormArgs& a, cudaStream_t s) {
  if (dtype == ATTAMBA_BF16)
    return res_dtype == ATTAMBA_BF16 ? launch_for<__nv_bfloat16, __nv_bfloat16>(a, s) : launch_for<__nv_bfloat16, float>(a, s);
  return res_dtype == ATTAMBA_BF16 ? launch_for<float, __nv_bfloat16>(a, s) : launch_for<float, float>(a, s);
}

}  // namespace attamba
