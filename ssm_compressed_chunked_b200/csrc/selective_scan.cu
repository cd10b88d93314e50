// Selective state-space scan over packed prompts with carried state, skip and gate,
// and its single-token step.
//
// Method: pith.science review of Attamba, "Assumptions & free parameters" -- Mamba's
// selective SSM (Section 3.2, Eq. 3).  Per token t, channel d:
//     delta = softplus(dt[t,d] + bias[d]);
//     h[:,d] = exp(delta A[d,:]) h[:,d] + delta x[t,d] B[t,:];
//     y[t,d] = (C[t,:] . h[:,d] + skip[d] x[t,d]) silu(z[t,d]).
//
// Split over time.  A sequence's tokens depend on one another through h alone, and
// h is linear in the h it starts from: over tokens a..b
//     h_b = exp(A sum_{a..b} delta) h_{a-1} + (h_b from h_{a-1} = 0).
// So the T token rows are cut into tiles that are scanned at once:
//   1. scan_tile<state pass>  per tile but the last: its end state from zero (or from
//      its sequence's own start, when that lies in the tile) and its sum of deltas;
//   2. scan_join              per (n, d): walks the tiles, each tile's end state in place;
//   3. scan_tile<output pass> per tile: from the end state of the tile before it.
// A tile that a sequence starts in takes the carried state in step 1 and keeps it for
// step 3, whose last tile of that sequence replaces the state row.  One tile needs
// step 3 alone.
#include "common.cuh"
#include "launch.h"

namespace attamba {

namespace {
constexpr int kThreads = 128;
constexpr int kStageTokens = 64;   // window of staged B and C rows

// CPT neighbouring channels of a token row
template <typename T, int CPT> struct Row;
template <> struct Row<__nv_bfloat16, 1> {
  using raw = unsigned short;
  static __device__ __forceinline__ void unpack(raw r, float (&v)[1]) { v[0] = __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ raw pack(const float (&v)[1]) { return __bfloat16_as_ushort(__float2bfloat16_rn(v[0])); }
};
template <> struct Row<__nv_bfloat16, 2> {
  using raw = uint32_t;
  static __device__ __forceinline__ void unpack(raw r, float (&v)[2]) {
    v[0] = __uint_as_float(r << 16);
    v[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ raw pack(const float (&v)[2]) { return pack_bf16x2(v[0], v[1]); }
};
template <> struct Row<float, 1> {
  using raw = float;
  static __device__ __forceinline__ void unpack(raw r, float (&v)[1]) { v[0] = r; }
  static __device__ __forceinline__ raw pack(const float (&v)[1]) { return v[0]; }
};
template <> struct Row<float, 2> {
  using raw = float2;
  static __device__ __forceinline__ void unpack(raw r, float (&v)[2]) { v[0] = r.x; v[1] = r.y; }
  static __device__ __forceinline__ raw pack(const float (&v)[2]) { return make_float2(v[0], v[1]); }
};

// Workspace: end states [tiles - 1, N, D], carried states of sequences that start in a tile and
// leave it [tiles - 1, N, D], sums of deltas [tiles - 1, D] (-1: the tile's end state is final).
struct ScanWork {
  float* end;
  float* kept;
  float* sum;
};
__host__ __device__ inline ScanWork scan_work(float* w, int tiles, int N, int D) {
  const size_t n = (size_t)(tiles - 1) * N * D;
  return {w, w + n, w + 2 * n};
}

// One block: kThreads / LPC * CPT channels of one tile.  LPC lanes share a channel, each with
// NS / LPC of its states; FULL: the output pass.
template <typename T, int CPT, int LPC, int NS, bool FULL, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) scan_tile_kernel(SelScanArgs p, int tile_len, int tiles) {
  using R = Row<T, CPT>;
  using raw = typename R::raw;
  constexpr int NPL = NS / LPC, NP = NPL / 2;
  __shared__ __align__(16) float sBC[kStageTokens][2 * NS];
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int lane = threadIdx.x & 31;
  const int groups = (p.D + kThreads / LPC * CPT - 1) / (kThreads / LPC * CPT);
  const int tile = blockIdx.x / groups, group = blockIdx.x % groups;
  const int64_t t0 = (int64_t)tile * tile_len;
  const bool last_tile = tile == tiles - 1;
  if (FULL && blockIdx.x == 0 && threadIdx.x < 32)
    check_sequences_warp(p.cu, p.S, p.T, lane, p.status);
  const int total = max(0, (int)min((int64_t)p.cu[p.S], p.T));
  const int t1 = (int)min(t0 + tile_len, (int64_t)total);
  const int D = p.D;
  const int c0 = (group * kThreads + (int)threadIdx.x) / LPC * CPT;
  const int n0 = (threadIdx.x % LPC) * NPL;
  const bool active = c0 < D;
  const ScanWork ws = scan_work(p.work, tiles, NS, D);

  float2 a2[CPT][NP], h[CPT][NP];
  float bias[CPT], skip[CPT], sum[CPT];
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    bias[c] = active && p.bias ? __ldg(p.bias + c0 + c) : 0.f;
    skip[c] = FULL && active && p.skip ? __ldg(p.skip + c0 + c) : 0.f;
    sum[c] = 0.f;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      float2 v = make_float2(0.f, 0.f);
      if (active) v = __ldg(reinterpret_cast<const float2*>(p.A + (size_t)(c0 + c) * NS + n0 + 2 * q));
      a2[c][q] = make_float2(v.x * kLog2e, v.y * kLog2e);
      h[c][q] = make_float2(0.f, 0.f);
    }
  }
  const T* __restrict__ x = static_cast<const T*>(p.x) + c0;
  const T* __restrict__ dt = static_cast<const T*>(p.dt) + c0;
  const T* __restrict__ z = static_cast<const T*>(p.z) + c0;
  const T* __restrict__ Bm = static_cast<const T*>(p.Bm);
  const T* __restrict__ Cm = static_cast<const T*>(p.Cm);
  T* __restrict__ y = static_cast<T*>(p.y) + c0;
  auto get = [&](const T* q, int t, int ld) { return __ldg(reinterpret_cast<const raw*>(q + (int64_t)t * ld)); };

  // state rows [NS, D]: this thread's CPT channels of its NPL states
  auto load_state = [&](const float* q) {
#pragma unroll
    for (int n = 0; n < NPL; ++n)
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        const float v = active ? q[(size_t)(n0 + n) * D + c0 + c] : 0.f;
        if (n & 1) h[c][n / 2].y = v;
        else h[c][n / 2].x = v;
      }
  };
  auto store_state = [&](float* q) {
    if (!active) return;
#pragma unroll
    for (int n = 0; n < NPL; ++n)
#pragma unroll
      for (int c = 0; c < CPT; ++c) q[(size_t)(n0 + n) * D + c0 + c] = (n & 1) ? h[c][n / 2].y : h[c][n / 2].x;
  };
  auto zero_state = [&]() {
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int q = 0; q < NP; ++q) h[c][q] = make_float2(0.f, 0.f);
  };

  // tokens [a, b), all of one sequence; by the whole block
  auto walk = [&](int a, int b) {
    const bool gated = FULL && p.z != nullptr;
    auto tok = [&](int t) { return min(t, b - 1); };   // harmless reloads past the end
    float dl[2][CPT], xv[2][CPT];
    raw rx[2] = {}, rd[2] = {}, rz[2] = {}, rg[2] = {};
    auto delta_of = [&](int j) {
      float v[CPT];
      R::unpack(rx[j], xv[j]);
      R::unpack(rd[j], v);
#pragma unroll
      for (int c = 0; c < CPT; ++c) dl[j][c] = softplus_f(v[c] + bias[c]);
      rg[j] = rz[j];
    };
    auto fetch = [&](int j, int t) {
      rx[j] = get(x, tok(t), p.ldx);
      rd[j] = get(dt, tok(t), p.lddt);
      if (gated) rz[j] = get(z, tok(t), p.ldz);
    };
    if (active) {
      fetch(0, a);
      fetch(1, a + 1);
      delta_of(0);
      delta_of(1);
      fetch(0, a + 2);
      fetch(1, a + 3);
    }
    auto step = [&](int t, int j, const float* bc) {
      float out[CPT];
      const float2* b2 = reinterpret_cast<const float2*>(bc + n0);
      const float2* c2 = reinterpret_cast<const float2*>(bc + NS + n0);
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        const float2 dl2 = make_float2(dl[j][c], dl[j][c]);
        const float dx = dl[j][c] * xv[j][c];
        const float2 dx2 = make_float2(dx, dx);
        float2 ya = make_float2(0.f, 0.f), yb = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          const float2 e = mul2(dl2, a2[c][q]);
          h[c][q] = fma2(make_float2(ex2(e.x), ex2(e.y)), h[c][q], mul2(dx2, b2[q]));
          if (FULL) {
            if (q & 1) yb = fma2(c2[q], h[c][q], yb);
            else ya = fma2(c2[q], h[c][q], ya);
          }
        }
        if (FULL) {
          float v = (ya.x + ya.y) + (yb.x + yb.y);
#pragma unroll
          for (int m = 1; m < LPC; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
          out[c] = fmaf(skip[c], xv[j][c], v);
        } else {
          sum[c] += dl[j][c];
        }
      }
      if (FULL) {
        if (gated) {
          float g[CPT];
          R::unpack(rg[j], g);
#pragma unroll
          for (int c = 0; c < CPT; ++c) out[c] *= silu_f(g[c]);
        }
        if (active && threadIdx.x % LPC == 0)
          *reinterpret_cast<raw*>(y + (int64_t)t * p.ldy) = R::pack(out);
      }
    };
    for (int tb = a; tb < b; tb += kStageTokens) {
      const int nt = min(kStageTokens, b - tb);
      __syncthreads();
      for (int e = threadIdx.x; e < nt * NS; e += kThreads) {
        const int k = e / NS, n = e - k * NS;
        sBC[k][n] = Elem<T>::to_f(Bm[(int64_t)(tb + k) * p.ldb + n]);
        if (FULL) sBC[k][NS + n] = Elem<T>::to_f(Cm[(int64_t)(tb + k) * p.ldc + n]);
      }
      __syncthreads();
      for (int k = 0; k < nt; k += 2) {
        const int t = tb + k;
        step(t, 0, &sBC[k][0]);
        if (k + 1 < nt) step(t + 1, 1, &sBC[k + 1][0]);
        if (active) {
          delta_of(0);
          delta_of(1);
          fetch(0, t + 4);
          fetch(1, t + 5);
        }
      }
    }
  };

  if (!FULL) {
    // the sequence that tokens t1 - 1 and t1 both belong to, if any: only its state leaves the tile
    float* sum_row = ws.sum + (size_t)tile * D;
    int first = t1;
    int s = 0;
    if (t0 + tile_len < total) {
      s = count_below_warp(p.cu, p.S, t1, lane) - 1;     // the last sequence that starts ahead of t1
      if (s >= 0 && p.cu[s + 1] > t1) first = max(0, p.cu[s]);
    }
    if (first >= t1) {
      if (active && threadIdx.x % LPC == 0)
        for (int c = 0; c < CPT; ++c) sum_row[c0 + c] = -1.f;
      return;
    }
    const bool starts = first >= t0;
    if (starts) {
      const int slot = p.state ? state_slot_warp(p.slots, s, p.n_slots, lane, p.status) : -1;
      if (slot >= 0 && p.cont && p.cont[s] != 0) {
        load_state(p.state + (size_t)slot * NS * D);
        store_state(ws.kept + (size_t)tile * NS * D);
      }
    }
    walk((int)max((int64_t)first, t0), t1);
    store_state(ws.end + (size_t)tile * NS * D);
    if (active && threadIdx.x % LPC == 0)
      for (int c = 0; c < CPT; ++c) sum_row[c0 + c] = starts ? -1.f : sum[c];
    return;
  }

  // the first sequence that starts in this tile; the one before it may reach into the tile
  int s = count_below_warp(p.cu, p.S, (int)t0, lane);
  if (s > 0 && tile > 0) {
    const int end = p.cu[s], b = min(end, t1);
    if (t0 < b) {
      load_state(ws.end + (size_t)(tile - 1) * NS * D);
      walk((int)t0, b);
      if (end <= t1 && p.state) {
        const int slot = state_slot_warp(p.slots, s - 1, p.n_slots, lane, p.status);
        if (slot >= 0) store_state(p.state + (size_t)slot * NS * D);
      }
    }
  }
  int t = (int)min(t0, (int64_t)total);
  for (; s < p.S; ++s) {
    const int cs = p.cu[s];
    if (cs >= t0 + tile_len && !last_tile) break;
    const int first = min(max(cs, t), total);             // clamps act on a malformed cu only
    const int end = min(max(p.cu[s + 1], first), total);
    const int slot = p.state ? state_slot_warp(p.slots, s, p.n_slots, lane, p.status) : -1;
    zero_state();
    if (slot >= 0 && p.cont && p.cont[s] != 0)
      load_state(end > t1 ? ws.kept + (size_t)tile * NS * D : p.state + (size_t)slot * NS * D);
    const int b = min(end, t1);
    if (first < b) walk(first, b);
    if (end <= t1 && slot >= 0) store_state(p.state + (size_t)slot * NS * D);
    t = max(t, b);
  }
}

// one thread per (n, d): end states of the tiles, in place
template <int NS>
__global__ void __launch_bounds__(kThreads) scan_join_kernel(SelScanArgs p, int tiles) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x * kThreads + threadIdx.x;   // n * D + d
  if (i >= NS * p.D) return;
  const int n = i / p.D, d = i - n * p.D;
  const ScanWork ws = scan_work(p.work, tiles, NS, p.D);
  const float a2 = p.A[(size_t)d * NS + n] * kLog2e;
  float h = 0.f;
  for (int k = 0; k + 1 < tiles; ++k) {
    const float sum = ws.sum[(size_t)k * p.D + d];
    float* e = ws.end + (size_t)k * NS * p.D + i;
    h = sum < 0.f ? *e : fmaf(ex2(a2 * sum), h, *e);
    *e = h;
  }
}

// Single-token step.  A warp has 32 channels of one batch row: lane = (state quarter, 4 channels), so
// its state accesses are 16 bytes a lane and a row of 128 bytes a quarter.
template <typename T, int NS>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(SelScanArgs p) {
  constexpr int NPL = NS / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x;
  const int slot = state_slot_warp(p.slots, b, p.n_slots, lane, p.status);
  if (slot < 0) return;
  const int c0 = ((int)blockIdx.y * (kThreads / 32) + warp) * 32 + (lane & 7) * 4;
  const int n0 = (lane >> 3) * NPL;
  const bool active = c0 < p.D;
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  float x[4], v[4];
  auto row4 = [&](const void* q, int ld, float (&o)[4]) {
    const T* r = static_cast<const T*>(q) + (int64_t)b * ld + c0;
    if (sizeof(T) == 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(r));
      o[0] = f.x; o[1] = f.y; o[2] = f.z; o[3] = f.w;
    } else {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(r));
      o[0] = __uint_as_float(u.x << 16); o[1] = __uint_as_float(u.x & 0xffff0000u);
      o[2] = __uint_as_float(u.y << 16); o[3] = __uint_as_float(u.y & 0xffff0000u);
    }
  };
  if (active) {
    float4* st = reinterpret_cast<float4*>(p.state + ((size_t)slot * NS + n0) * p.D + c0);
    const size_t ld4 = (size_t)p.D / 4;
    float4 h[NPL];
#pragma unroll
    for (int n = 0; n < NPL; ++n) h[n] = st[n * ld4];
    row4(p.x, p.ldx, x);
    row4(p.dt, p.lddt, v);
    float dl[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) dl[c] = softplus_f(v[c] + (p.bias ? __ldg(p.bias + c0 + c) : 0.f));
    const T* Bm = static_cast<const T*>(p.Bm) + (int64_t)b * p.ldb + n0;
    const T* Cm = static_cast<const T*>(p.Cm) + (int64_t)b * p.ldc + n0;
#pragma unroll
    for (int n = 0; n < NPL; ++n) {
      const float Bn = Elem<T>::to_f(Bm[n]), Cn = Elem<T>::to_f(Cm[n]);
      float* hn = reinterpret_cast<float*>(&h[n]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float a = __ldg(p.A + (size_t)(c0 + c) * NS + n0 + n) * kLog2e;
        hn[c] = fmaf(ex2(dl[c] * a), hn[c], dl[c] * x[c] * Bn);
        y[c] = fmaf(Cn, hn[c], y[c]);
      }
    }
#pragma unroll
    for (int n = 0; n < NPL; ++n) st[n * ld4] = h[n];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    y[c] += __shfl_xor_sync(0xffffffffu, y[c], 8);
    y[c] += __shfl_xor_sync(0xffffffffu, y[c], 16);
  }
  if (active && n0 == 0) {
    if (p.skip) {
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] = fmaf(__ldg(p.skip + c0 + c), x[c], y[c]);
    }
    if (p.z) {
      row4(p.z, p.ldz, v);
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] *= silu_f(v[c]);
    }
    T* o = static_cast<T*>(p.y) + (int64_t)b * p.ldy + c0;
    if (sizeof(T) == 4) *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
    else *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  }
}

// Tokens per tile.
int scan_tile_len(int64_t T) { return 128; }

template <typename T, int NS>
cudaError_t launch_scan(const SelScanArgs& a, cudaStream_t s) {
  constexpr int CPT = NS == 16 ? 2 : 1;
  const int len = scan_tile_len(a.T);
  const int tiles = (int)((a.T + len - 1) / len);
  const int64_t groups = (a.D + kThreads * CPT - 1) / (kThreads * CPT);
  if (groups * tiles > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e;
  if (tiles > 1) {
    e = launch_dependent(scan_tile_kernel<T, CPT, 1, NS, false, 3>, dim3((unsigned)(groups * (tiles - 1))), kThreads, s, a, len, tiles);
    if (e != cudaSuccess) return e;
    e = launch_dependent(scan_join_kernel<NS>, dim3((NS * a.D + kThreads - 1) / kThreads), kThreads, s, a, tiles);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(scan_tile_kernel<T, CPT, 1, NS, true, 3>, dim3((unsigned)(groups * tiles)), kThreads, s, a, len, tiles);
}

template <typename T, int NS>
cudaError_t launch_step(const SelScanArgs& a, cudaStream_t s) {
  return launch_dependent(scan_step_kernel<T, NS>, dim3((unsigned)a.T, (a.D + kThreads - 1) / kThreads), kThreads, s, a);
}
}  // namespace

size_t selective_scan_workspace_bytes(int64_t T, int32_t D, int32_t N) {
  const int len = scan_tile_len(T);
  const int64_t tiles = (T + len - 1) / len;
  return (size_t)(tiles - 1) * D * (2 * N + 1) * sizeof(float);
}

cudaError_t launch_selective_scan(attamba_dtype_t dtype, const SelScanArgs& a, cudaStream_t s) {
  if (dtype == ATTAMBA_BF16)
    return a.N == 16 ? launch_scan<__nv_bfloat16, 16>(a, s) : launch_scan<__nv_bfloat16, 32>(a, s);
  return a.N == 16 ? launch_scan<float, 16>(a, s) : launch_scan<float, 32>(a, s);
}

cudaError_t launch_scan_step(attamba_dtype_t dtype, const SelScanArgs& a, cudaStream_t s) {
  if (dtype == ATTAMBA_BF16)
    return a.N == 16 ? launch_step<__nv_bfloat16, 16>(a, s) : launch_step<__nv_bfloat16, 32>(a, s);
  return a.N == 16 ? launch_step<float, 16>(a, s) : launch_step<float, 32>(a, s);
}

}  // namespace attamba
