// Device helpers of the SSM block's operators: activations, state slots and sequence tables, asynchronous copies.
// What these kernels share with the others is in common.cuh.
#pragma once

#include "common.cuh"

namespace attamba {

// ---------------------------------------------------------------- arithmetic
// softplus_f of a pair, the same steps two wide
__device__ __forceinline__ float2 softplus2(float2 z) {
  const float2 one = make_float2(1.f, 1.f);
  const float2 e = mul2(z, make_float2(kLog2e, kLog2e));
  const float2 u = make_float2(ex2(e.x), ex2(e.y)), w = add2(one, u);
  float2 lg;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg.x) : "f"(w.x));
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg.y) : "f"(w.y));
  lg = mul2(lg, make_float2(0.6931471805599453f, 0.6931471805599453f));
  float2 s = fma2(u, make_float2(0.2f, 0.2f), make_float2(-0.25f, -0.25f));
  s = fma2(u, s, make_float2(1.f / 3.f, 1.f / 3.f));
  s = fma2(u, s, make_float2(-0.5f, -0.5f));
  s = mul2(u, fma2(u, s, one));
  const float a = u.x < 0.0625f ? s.x : lg.x, b = u.y < 0.0625f ? s.y : lg.y;
  return make_float2(z.x > 20.f ? z.x : a, z.y > 20.f ? z.y : b);
}

// 1 / (1 + e^-z) and silu(z) = z / (1 + e^-z), with the hardware's reciprocal (2^-23 of the value).  e^-z overflows
// to infinity for z < -88.7, its reciprocal is then 0.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid_f(float z) { return rcp(1.f + ex2(-z * kLog2e)); }
__device__ __forceinline__ float silu_f(float z) { return z * sigmoid_f(z); }
__device__ __forceinline__ float2 silu2(float2 z) {
  const float2 e = mul2(z, make_float2(-kLog2e, -kLog2e));
  const float2 d = add2(make_float2(ex2(e.x), ex2(e.y)), make_float2(1.f, 1.f));
  return mul2(z, make_float2(rcp(d.x), rcp(d.y)));
}

// ---------------------------------------------------------------- slots and sequence tables
// Whether sequence (or batch row) s may use its state row: the slot lies in [0, n_slots) and no earlier
// one has it.  By all 32 lanes; a wrong slot raises ATTAMBA_DEV_BAD_SEQS.  Returns the slot, or -1.
__device__ __forceinline__ int state_slot_warp(const int32_t* slots, int s, int n_slots, int lane, int32_t* st) {
  const int slot = slots ? __ldg(slots + s) : s;
  if (slot == -1) return -1;
  bool bad = slot < 0 || slot >= n_slots;
  if (slots && !bad) {
#pragma unroll 8
    for (int i = lane; i < s; i += 32) bad |= __ldg(slots + i) == slot;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) raise_status(st, ATTAMBA_DEV_BAD_SEQS);
    return -1;
  }
  return slot;
}

// state_slot_warp for up to 32 batch rows first, first + stride, ... < rows at once, by a whole block: lane j of every
// warp gets row j's answer.  The rows' slots go into a small hash table (a bit per row); each slot ahead of the last row
// then costs one look-up, however many rows there are.
struct SlotTable {
  static constexpr int kEntries = 256;
  uint32_t rows[kEntries];   // by slot mod kEntries: which rows have such a slot
  int slot[32];
  uint32_t repeated;
};
__device__ __forceinline__ int state_slots_block(const int32_t* slots, int first, int stride, int rows, int n_slots,
                                                 SlotTable& t, int32_t* st) {
  const int lane = threadIdx.x & 31;
  const int64_t mine = first + (int64_t)lane * stride;
  int slot = mine < rows ? (slots ? __ldg(slots + mine) : (int)mine) : -1;
  bool bad = slot != -1 && (slot < 0 || slot >= n_slots);
  if (slots) {
    const int n = min(32, (rows - first + stride - 1) / stride);
    const int last = first + (n - 1) * stride;   // slots[0, last) lie ahead of some row
    __syncthreads();                             // the table's last use is over
    for (int i = threadIdx.x; i < SlotTable::kEntries; i += blockDim.x) t.rows[i] = 0;
    if (threadIdx.x == 0) t.repeated = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
      t.slot[lane] = slot;
      if (slot >= 0) atomicOr(&t.rows[slot % SlotTable::kEntries], 1u << lane);
    }
    __syncthreads();
#pragma unroll 4
    for (int j = threadIdx.x; j < last; j += blockDim.x) {
      const int v = __ldg(slots + j);
      uint32_t m = v >= 0 ? t.rows[v % SlotTable::kEntries] : 0;
      while (m) {
        const int i = __ffs(m) - 1;
        m &= m - 1;
        if (t.slot[i] == v && j < first + i * stride) atomicOr(&t.repeated, 1u << i);
      }
    }
    __syncthreads();
    bad |= slot != -1 && ((t.repeated >> lane) & 1);
  }
  if (bad) {
    if (threadIdx.x < 32) raise_status(st, ATTAMBA_DEV_BAD_SEQS);
    slot = -1;
  }
  return slot;
}

// Whether cu[0, S] is 0 = cu[0] <= ... <= cu[S] <= T; by one warp.
__device__ __forceinline__ void check_sequences_warp(const int32_t* cu, int S, int64_t T, int lane, int32_t* st) {
  bool bad = cu[0] != 0 || cu[S] > T;
  for (int i = lane; i < S; i += 32) bad |= cu[i] > cu[i + 1];
  if (__any_sync(0xffffffffu, bad) && lane == 0) raise_status(st, ATTAMBA_DEV_BAD_SEQS);
}

// ---------------------------------------------------------------- asynchronous copies
// asynchronous copies of 8 or 16 bytes, global to shared, and the thread's groups of them
template <int BYTES> __device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace attamba
