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
// step 3 alone.  Steps 2 and 3 are programmatic dependents: their blocks are placed and
// step 3's first windows loaded while the step before drains.
//
// Mapping (B200).  A block has the channels of 128 / LPC * CPT threads and walks its tile
// token by token, the state and A log2 e in registers as f32x2 pairs over n.  x, dt and z
// come in windows of 12 bf16 rows by cp.async, one window ahead; B and C, the same for
// all channels, are staged as fp32 and read as broadcast 16-byte loads.  The loop is
// independent of the sequences: a window is walked in runs that end where one does.
//
// What bounds it: the exponentials.  Both passes take T D N of them, on a unit that does
// 16 a clock and SM, beside 4 (output) or 3 (state) half-rate f32x2 operations a pair: at
// 16384 x 1024 x 16 (bf16, gated) that is 60 + 67 us at 1.9 GHz, and the call takes 176
// (0.77 TB/s of 6.47): K tiles take the exponentials 2 - 1/K times, and K is 110 here.  The unit is
// 82% busy in the state pass, 69% in the output pass, the issue slots 43 and 46%; three warps a scheduler
// is what the registers hold.  Measured and not kept: one channel a thread and five to seven blocks on an SM
// (196-221 us), two channels at four blocks (194), three quarters of the window (186),
// all groups of a window unrolled (185), the short batches' tiles as a cluster that exchanges
// states through distributed shared memory (61 tokens 9.9 us against 6.9 in a single tile).
#include <type_traits>

#include "launch.h"
#include "ssm_block.cuh"

namespace attamba {

namespace {
constexpr int kThreads = 128;
constexpr int kWindowBytes = 24;   // a window's tokens times the element's size: 12 bf16 or 6 f32 tokens
constexpr int kStages = 2;         // windows of x, dt and z in shared memory
// 2^f = 1 + f (kE1 + f (kE2 + ...)) on [-1/2, 1/2], fitted by linear programming for the least largest relative error
// (9.2e-8): relative error 1.1e-7 with the coefficients rounded to fp32, 1.75e-7 once the sums are rounded, unbiased near 0
constexpr float kE1 = 0.6931470036506653f, kE2 = 0.24022242426872253f, kE3 = 0.05550733953714371f,
                kE4 = 0.009671511128544807f, kE5 = 0.0013264646986499429f;

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

// 2^x for the x = dl a of a decay, on the FMA pipe: x = j + f with j the nearest integer, 2^f by a polynomial
// with p(0) = 1, j added to the exponent field.  x is clamped at -126, where 2^x ends as the smallest normal
// number (the hardware's instruction flushes what is below it to zero).
__device__ __forceinline__ float2 decay_fma2(float2 dl, float2 a) {
  const float2 magic = make_float2(12582912.f, 12582912.f);   // 1.5 * 2^23
  const float2 x0 = mul2(dl, a);
  const float2 x = make_float2(fmaxf(x0.x, -126.f), fmaxf(x0.y, -126.f));
  const float2 t = add2(x, magic);
  const float2 f = sub2(x, sub2(t, magic));
  float2 q = fma2(f, make_float2(kE5, kE5), make_float2(kE4, kE4));
  q = fma2(q, f, make_float2(kE3, kE3));
  q = fma2(q, f, make_float2(kE2, kE2));
  q = fma2(q, f, make_float2(kE1, kE1));
  q = fma2(q, f, make_float2(1.f, 1.f));
  return make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + __float_as_uint(q.x)),
                     __uint_as_float((__float_as_uint(t.y) << 23) + __float_as_uint(q.y)));
}

// One block: kThreads / LPC * CPT channels of one tile.  LPC lanes share a channel, each with
// NS / LPC of its states; FULL: the output pass.
template <typename T, int CPT, int LPC, int NS, bool FULL, int MINB, int POLY>
__global__ void __launch_bounds__(kThreads, MINB) scan_tile_kernel(SelScanArgs p, int tile_len, int tiles) {
  using R = Row<T, CPT>;
  using raw = typename R::raw;
  constexpr int NPL = NS / LPC, NP = NPL / 2;
  constexpr int GT = LPC > 1 ? LPC : 2, TPL = GT / LPC;   // tokens of a group, and of them a lane's
  constexpr int W = (kWindowBytes / (int)sizeof(T) + GT - 1) / GT * GT;   // tokens per window
  constexpr int CB = kThreads / LPC * CPT;                // channels per block
  constexpr int kArrays = FULL ? 3 : 2;                   // x, dt and z
  constexpr int kBC = FULL ? 2 * NS : NS;
  constexpr int kBCPer = (W * kBC + kThreads - 1) / kThreads;
  __shared__ __align__(16) T sRow[kStages][kArrays][W][CB];
  __shared__ __align__(16) float sBC[2][W][kBC];
  // The output pass after a state pass reads nothing the kernels between them and it write until it needs the
  // carried state (below): its first loads overlap their end.
  if (!FULL || tiles == 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!FULL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int lane = threadIdx.x & 31;
  const int groups = (p.D + CB - 1) / CB;
  const int tile = blockIdx.x / groups, group = blockIdx.x % groups;
  const int64_t t0 = (int64_t)tile * tile_len;
  const bool last_tile = tile == tiles - 1;
  if (FULL && blockIdx.x == 0 && threadIdx.x < 32)
    check_sequences_warp(p.cu, p.S, p.T, lane, p.status);
  const int total = max(0, (int)min((int64_t)p.cu[p.S], p.T));
  const int t1 = (int)min(t0 + tile_len, (int64_t)total);
  const int D = p.D;
  const int cb = group * CB;                              // the block's first channel
  const int cl = threadIdx.x / LPC * CPT;                 // this thread's, in the block
  const int c0 = cb + cl;
  const int part = threadIdx.x % LPC;                     // and its share of the states
  const int n0 = part * NPL;
  const bool active = c0 < D;
  const bool gated = FULL && p.z != nullptr;
  const ScanWork ws = scan_work(p.work, tiles, NS, D);

  // the tokens this block walks: its tile, or in the state pass the part of it that the state leaving it hangs on
  int first = (int)min(t0, (int64_t)total);
  int seq = 0;
  if (!FULL) {
    first = t1;
    if (t0 + tile_len < total) {
      seq = count_below_warp(p.cu, p.S, t1, lane) - 1;   // the last sequence that starts ahead of t1
      if (seq >= 0 && p.cu[seq + 1] > t1) first = max(0, p.cu[seq]);
    }
    if (first >= t1) {   // no sequence reaches from this tile into the next
      if (active && threadIdx.x % LPC == 0)
        for (int c = 0; c < CPT; ++c) ws.sum[(size_t)tile * D + c0 + c] = -1.f;
      return;
    }
  }
  const bool starts = !FULL && first >= t0;
  const int w0 = FULL ? first : (int)max((int64_t)first, t0);   // first token of window 0
  const int windows = t1 > w0 ? (t1 - w0 + W - 1) / W : 0;

  // window k: x, dt, z into stage k % kStages; B, C through registers, as fp32, into sBC[k % 2].  A thread copies
  // the same 16-byte column of every kRowStep-th row; its addresses move on by a window a call.
  constexpr int kCols = CB * (int)sizeof(T) / 16, kRowStep = kThreads / kCols > 0 ? kThreads / kCols : 1;
  static_assert(kCols <= kThreads, "a row of a window is at most a piece a thread");
  const int crow = threadIdx.x / kCols, ccol = threadIdx.x % kCols * (16 / (int)sizeof(T));
  const bool copies = cb + ccol < D;
  const T* px = static_cast<const T*>(p.x) + (int64_t)(w0 + crow) * p.ldx + cb + ccol;
  const T* pdt = static_cast<const T*>(p.dt) + (int64_t)(w0 + crow) * p.lddt + cb + ccol;
  const T* pz = static_cast<const T*>(p.z) + (int64_t)(w0 + crow) * p.ldz + cb + ccol;
  auto load_rows = [&](int k) {
    const int left = t1 - w0 - k * W;   // tokens of the tile from this window on
    T* dst = &sRow[k % kStages][0][crow][ccol];
#pragma unroll
    for (int r = 0; r < W; r += kRowStep) {
      if ((W % kRowStep == 0 || crow + r < W) && crow + r < left && copies) {
        copy_async<16>(dst + r * CB, px + (int64_t)r * p.ldx);
        copy_async<16>(dst + (W + r) * CB, pdt + (int64_t)r * p.lddt);
        if (gated) copy_async<16>(dst + (2 * W + r) * CB, pz + (int64_t)r * p.ldz);
      }
    }
    px += (int64_t)W * p.ldx;
    pdt += (int64_t)W * p.lddt;
    pz += (int64_t)W * p.ldz;
    copies_commit();   // a group per window, empty ones too: the wait counts groups
  };
  T bc[kBCPer];   // converted when stored: the conversion would wait for the load
  auto load_bc = [&](int k) {
#pragma unroll
    for (int i = 0; i < kBCPer; ++i) {
      const int e = threadIdx.x + i * kThreads;
      const int row = e / kBC, n = e % kBC;
      const int tk = w0 + k * W + row;
      bc[i] = T(0.f);
      if (e < W * kBC && tk < t1 && k < windows)
        bc[i] = n < NS ? static_cast<const T*>(p.Bm)[(int64_t)tk * p.ldb + n]
                       : static_cast<const T*>(p.Cm)[(int64_t)tk * p.ldc + n - NS];
    }
  };
  auto store_bc = [&](int k) {
#pragma unroll
    for (int i = 0; i < kBCPer; ++i) {
      const int e = threadIdx.x + i * kThreads;
      if (e < W * kBC) (&sBC[k % 2][0][0])[e] = Elem<T>::to_f(bc[i]);
    }
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) load_rows(k);
  load_bc(0);
  store_bc(0);
  load_bc(1);

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
  T* __restrict__ y = static_cast<T*>(p.y) + c0;

  // state rows [NS, D]: this thread's CPT channels of its NPL states
  // (a state row lies in the state array: state_slot_warp; an end state and a kept one in the workspace: tile < tiles - 1)
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

  int window = -1;   // the window in shared memory that the walk has reached
  // tokens [a, b), all of one sequence, next to those walked before; by the whole block
  auto walk = [&](int a, int b) {
    if (!in_bounds(a >= w0 && b <= t1 && t1 <= p.T, p.status)) return;   // the same for every thread
    // decay_fma2 makes a number of a NaN; one in A reaches the state here (one in delta through delta x B)
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int q = 0; q < POLY; ++q) {
        if (isnan(a2[c][q].x)) h[c][q].x = a2[c][q].x;
        if (isnan(a2[c][q].y)) h[c][q].y = a2[c][q].y;
      }
    for (int t = a; t < b;) {
      const int k = (t - w0) / W;
      if (k != window) {
        window = k;
        copies_wait<kStages - 2>();
        __syncthreads();               // window k has arrived for all, window k - 1 has been read by all
        load_rows(k + kStages - 1);
        store_bc(k + 1);
        load_bc(k + 2);
      }
      const int r0 = t - w0 - k * W, r1 = min(b - w0 - k * W, W);
      const T* rx = &sRow[k % kStages][0][0][cl];
      const float* rbc = &sBC[k % 2][0][n0];
      // group of GT tokens: token j is prepared and finished by lane j % LPC of its channels' lanes
      float xv[TPL][CPT], dl[TPL][CPT];
      auto prepare = [&](int g) {
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
          const int r = min(g * GT + i * LPC + part, W - 1);   // past the window: not used
          float v[CPT];
          R::unpack(*reinterpret_cast<const raw*>(rx + r * CB), xv[i]);
          R::unpack(*reinterpret_cast<const raw*>(rx + (W + r) * CB), v);
          if (CPT == 2) {
            const float2 d = softplus2(make_float2(v[0] + bias[0], v[CPT - 1] + bias[CPT - 1]));
            dl[i][0] = d.x;
            dl[i][CPT - 1] = d.y;
          } else {
            dl[i][0] = softplus_f(v[0] + bias[0]);
          }
        }
      };
      auto group = [&](int g, auto whole) {
        constexpr bool kWhole = decltype(whole)::value;   // all GT tokens lie in [r0, r1)
        float part_y[GT][CPT], dcur[TPL][CPT], xcur[TPL][CPT];
#pragma unroll
        for (int i = 0; i < TPL; ++i)
#pragma unroll
          for (int c = 0; c < CPT; ++c) {
            dcur[i][c] = dl[i][c];
            xcur[i][c] = xv[i][c];
          }
#pragma unroll
        for (int j = 0; j < GT; ++j) {
          const int r = g * GT + j;
          const float2* b2 = reinterpret_cast<const float2*>(rbc + r * kBC);
          const float2* c2 = reinterpret_cast<const float2*>(rbc + r * kBC + NS);
          if (kWhole || (r >= r0 && r < r1)) {
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
              float d = dcur[j / LPC][c], dx = dcur[j / LPC][c] * xcur[j / LPC][c];
              if (LPC > 1) {
                d = __shfl_sync(0xffffffffu, d, j % LPC, LPC);
                dx = __shfl_sync(0xffffffffu, dx, j % LPC, LPC);
              }
              const float2 dl2 = make_float2(d, d), dx2 = make_float2(dx, dx);
              float2 ya = make_float2(0.f, 0.f), yb = make_float2(0.f, 0.f);
#pragma unroll
              for (int q = 0; q < NP; ++q) {
                float2 a;
                if (q < POLY) {
                  a = decay_fma2(dl2, a2[c][q]);
                } else {
                  const float2 e = mul2(dl2, a2[c][q]);
                  a = make_float2(ex2(e.x), ex2(e.y));
                }
                h[c][q] = fma2(a, h[c][q], mul2(dx2, b2[q]));
                if (FULL) {
                  if (q & 1) yb = fma2(c2[q], h[c][q], yb);
                  else ya = q == 0 ? mul2(c2[q], h[c][q]) : fma2(c2[q], h[c][q], ya);
                }
              }
              if (FULL) {
                if (NP > 1) ya = add2(ya, yb);
                part_y[j][c] = ya.x + ya.y;
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < CPT; ++c) part_y[j][c] = 0.f;
          }
        }
        prepare(g + 1);
        if (FULL) {
          // sum over the lanes, halving the tokens a lane holds at each step: lane q ends with tokens j % LPC == q
#pragma unroll
          for (int m = LPC / 2; m > 0; m /= 2) {
            const bool up = (part & m) != 0;
#pragma unroll
            for (int i = 0; i < GT / LPC; ++i)
#pragma unroll
              for (int u = 0; u < m; ++u)
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                  float& lo = part_y[i * LPC + u][c];
                  const float hi = part_y[i * LPC + u + m][c];
                  const float give = up ? lo : hi;
                  lo = (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, give, m);
                }
          }
#pragma unroll
          for (int i = 0; i < TPL; ++i) {
            const int r = g * GT + i * LPC + part;
            float out[CPT];
#pragma unroll
            for (int c = 0; c < CPT; ++c) out[c] = fmaf(skip[c], xcur[i][c], part_y[i * LPC][c]);
            if (gated) {
              float z[CPT];
              R::unpack(*reinterpret_cast<const raw*>(rx + (2 * W + r) * CB), z);
              if (CPT == 2) {
                const float2 g = silu2(make_float2(z[0], z[CPT - 1]));
                out[0] *= g.x;
                out[CPT - 1] *= g.y;
              } else {
                out[0] *= silu_f(z[0]);
              }
            }
            if (active && (kWhole || (r >= r0 && r < r1)))
              *reinterpret_cast<raw*>(y + (int64_t)(w0 + k * W + r) * p.ldy) = R::pack(out);
          }
        } else {
#pragma unroll
          for (int i = 0; i < TPL; ++i) {
            const int r = g * GT + i * LPC + part;
            if (kWhole || (r >= r0 && r < r1)) {
#pragma unroll
              for (int c = 0; c < CPT; ++c) sum[c] += dcur[i][c];
            }
          }
        }
      };
      prepare(r0 / GT);
      if (r0 == 0 && r1 == W) {
#pragma unroll 2
        for (int g = 0; g < W / GT; ++g) group(g, std::true_type{});
      } else {
#pragma unroll 1
        for (int g = r0 / GT; g * GT < r1; ++g) {
          if (g * GT >= r0 && (g + 1) * GT <= r1) group(g, std::true_type{});
          else group(g, std::false_type{});
        }
      }
      t = w0 + k * W + r1;
    }
  };

  if (!FULL) {
    if (starts) {
      const int slot = p.state ? state_slot_warp(p.slots, seq, p.n_slots, lane, p.status) : -1;
      if (slot >= 0 && p.cont && p.cont[seq] != 0) {
        load_state(p.state + (size_t)slot * NS * D);
        store_state(ws.kept + (size_t)tile * NS * D);
      }
    }
    walk(w0, t1);
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int m = 1; m < LPC; m *= 2) sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], m);
    store_state(ws.end + (size_t)tile * NS * D);
    if (active && threadIdx.x % LPC == 0)
      for (int c = 0; c < CPT; ++c) ws.sum[(size_t)tile * D + c0 + c] = starts ? -1.f : sum[c];
    return;
  }

  // the first sequence that starts in this tile; the one before it may reach into the tile
  int s = count_below_warp(p.cu, p.S, (int)t0, lane);
  int t = w0;
  if (tiles > 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (s > 0 && tile > 0) {
    const int end = p.cu[s], b = min(end, t1);
    if (t0 < b) {
      if (in_bounds(tile - 1 < tiles - 1, p.status)) load_state(ws.end + (size_t)(tile - 1) * NS * D);
      walk((int)t0, b);
      t = b;
      if (end <= t1 && p.state) {
        const int slot = state_slot_warp(p.slots, s - 1, p.n_slots, lane, p.status);
        if (slot >= 0) store_state(p.state + (size_t)slot * NS * D);
      }
    }
  }
  for (; s < p.S; ++s) {
    const int cs = p.cu[s];
    if (cs >= t0 + tile_len && !last_tile) break;
    const int from = min(max(cs, t), total);              // clamps act on a malformed cu only
    const int end = min(max(p.cu[s + 1], from), total);
    const int slot = p.state ? state_slot_warp(p.slots, s, p.n_slots, lane, p.status) : -1;
    zero_state();
    if (slot >= 0 && p.cont && p.cont[s] != 0 && in_bounds(end <= t1 || tile < tiles - 1, p.status))
      load_state(end > t1 ? ws.kept + (size_t)tile * NS * D : p.state + (size_t)slot * NS * D);
    const int b = min(end, t1);
    if (from < b) walk(from, b);
    if (end <= t1 && slot >= 0) store_state(p.state + (size_t)slot * NS * D);
    t = max(t, b);
  }
  copies_wait<0>();
}

// End states of the tiles, in place.  A block has 32 columns (n, d) and up to kJoinWarps runs of kJoin tiles: every
// warp joins its run from zero, the runs' (decay, state) pairs meet in shared memory, and each thread walks
// its run again from the state ahead of it.  The tiles' values stay in registers: one memory latency
// for kJoin * kJoinWarps tiles.
constexpr int kJoin = 8, kJoinWarps = 16;
template <int NS>
__global__ void __launch_bounds__(32 * kJoinWarps) scan_join_kernel(SelScanArgs p, int tiles) {
  __shared__ float sDecay[kJoinWarps][32], sEnd[kJoinWarps][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int i = blockIdx.x * 32 + lane;   // n * D + d; NS * D is a multiple of 32
  const int n = i / p.D, d = i - n * p.D;
  const ScanWork ws = scan_work(p.work, tiles, NS, p.D);
  const float a2 = p.A[(size_t)d * NS + n] * kLog2e;
  const size_t ld = (size_t)NS * p.D;
  float carry = 0.f;
  for (int k0 = 0; k0 + 1 < tiles; k0 += kJoin * warps) {
    const int k = k0 + warp * kJoin;
    float sum[kJoin], e[kJoin];
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const bool in = k + j + 1 < tiles;
      sum[j] = in ? ws.sum[(size_t)(k + j) * p.D + d] : -1.f;
      e[j] = in ? ws.end[(k + j) * ld + i] : 0.f;
    }
    float decay = 1.f, h = 0.f;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const bool fresh = sum[j] < 0.f;          // this tile's end state owes nothing to the tile ahead
      sum[j] = fresh ? -1.f : ex2(a2 * sum[j]);   // from here on its decay
      h = fresh ? e[j] : fmaf(sum[j], h, e[j]);
      decay = fresh ? -1.f : (decay < 0.f ? decay : decay * sum[j]);
    }
    sDecay[warp][lane] = decay;
    sEnd[warp][lane] = h;
    __syncthreads();
    h = carry;
    for (int w = 0; w < warps; ++w) {
      if (w == warp) carry = h;                 // the state ahead of this warp's run
      h = sDecay[w][lane] < 0.f ? sEnd[w][lane] : fmaf(sDecay[w][lane], h, sEnd[w][lane]);
    }
    float s = carry;
    carry = h;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      s = sum[j] < 0.f ? e[j] : fmaf(sum[j], s, e[j]);
      if (k + j + 1 < tiles) ws.end[(k + j) * ld + i] = s;
    }
    __syncthreads();                            // the pairs have been read
  }
}

// Single-token step.  A warp has 32 channels of a batch row: lane = (quarter of the states, 4 channels), so its
// state accesses are 16 bytes a lane, 128 bytes of a state row a quarter.  A block walks several batch rows of its
// 128 channels: A stays in registers, each thread copies its part of the next row's state into a ring of its own
// (cp.async, no barrier) and loads the next row's inputs while it computes this one's.  Bound by reading and writing
// the state: 251 rows x 2048 channels x 16 in 16.2-16.6 us (4.2 TB/s), 1024 rows in 53 (5.4), 256 x 4096 x 16 in 28 (5.2),
// x 32 in 52 (5.3): with five rows a block the ring's fill and drain are a third of the call (a copy of these rows in the same
// pattern takes 14.9); states that stay in the L2 take 11.8.  One row a block with everything in registers: 18.1 and 60.  The search for
// repeated slots (a hash table of the block's rows): 4096 x 1024 x 16 in 113 us, 91 without a slot map, 188 with
// every row compared with every slot ahead of it.
template <typename T> struct Four;
template <> struct Four<float> {
  using raw = float4;
  static __device__ __forceinline__ void unpack(const raw& f, float (&v)[4]) { v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w; }
};
template <> struct Four<__nv_bfloat16> {
  using raw = uint2;
  static __device__ __forceinline__ void unpack(const raw& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
  }
};
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <typename T> __device__ __forceinline__ typename Four<T>::raw get4(const void* p, int64_t at) {
  return __ldg(reinterpret_cast<const typename Four<T>::raw*>(static_cast<const T*>(p) + at));
}

constexpr int kStepDepth = 2;                                                  // batch rows in a thread's ring
constexpr int step_blocks(int NS) { return NS == 16 ? 6 : 3; }   // blocks on an SM: 7 or 8 spill and measured slower
template <typename T, int NS>
__global__ void __launch_bounds__(kThreads, step_blocks(NS)) scan_step_kernel(SelScanArgs p, int groups) {
  constexpr int NPL = NS / 4;
  __shared__ __align__(16) float4 ring[kStepDepth][NPL][kThreads];
  __shared__ SlotTable table;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = (((int)blockIdx.x % groups) * (kThreads / 32) + warp) * 32 + (lane & 7) * 4;
  const int n0 = (lane >> 3) * NPL;
  const bool active = c0 < p.D;
  const int first = blockIdx.x / groups, stride = gridDim.x / groups;   // this block's batch rows
  const int rows = (int)p.T;
  const size_t ld4 = (size_t)p.D / 4;
  auto state_of = [&](int slot) {
    return reinterpret_cast<float4*>(p.state + ((size_t)slot * NS + n0) * p.D + c0);
  };
  // a row's state on its way to the ring; a slot in range is safe to read before it is known to be good
  auto fetch = [&](int i) {
    const int b = first + i * stride;
    if (b < rows && active) {
      const int slot = p.slots ? __ldg(p.slots + b) : b;
      if (slot >= 0 && slot < p.n_slots) {
        const float4* st = state_of(slot);
#pragma unroll
        for (int n = 0; n < NPL; ++n) copy_async<16>(&ring[i % kStepDepth][n][threadIdx.x], st + n * ld4);
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kStepDepth - 1; ++i) fetch(i);
  // This lane prepares (softplus) and finishes (skip, gate) one of the four channels.
  const int oc = lane >> 3;
  float2 A[NPL][2];   // A log2 e of state n0 + n: channels 0, 1 and 2, 3
  float bias = 0.f, skip = 0.f;
  if (active) {
    if (p.bias) bias = __ldg(p.bias + c0 + oc);
    if (p.skip) skip = __ldg(p.skip + c0 + oc);
#pragma unroll
    for (int n = 0; n < NPL; n += 4) {
      float f[4][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) Four<float>::unpack(get4<float>(p.A, (int64_t)(c0 + c) * NS + n0 + n), f[c]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        A[n + k][0] = make_float2(f[0][k] * kLog2e, f[1][k] * kLog2e);
        A[n + k][1] = make_float2(f[2][k] * kLog2e, f[3][k] * kLog2e);
      }
    }
  }
  // a row's inputs, loaded one row ahead of their use
  using raw = typename Four<T>::raw;
  raw rx = {}, rB[NPL / 4] = {}, rC[NPL / 4] = {};
  T rdt = T(0.f), rz = T(0.f);
  auto load = [&](int b) {
    if (b >= rows || !active) return;
    rx = get4<T>(p.x, (int64_t)b * p.ldx + c0);
    rdt = static_cast<const T*>(p.dt)[(int64_t)b * p.lddt + c0 + oc];
    if (p.z) rz = static_cast<const T*>(p.z)[(int64_t)b * p.ldz + c0 + oc];
#pragma unroll
    for (int n = 0; n < NPL / 4; ++n) {
      rB[n] = get4<T>(p.Bm, (int64_t)b * p.ldb + n0 + 4 * n);
      rC[n] = get4<T>(p.Cm, (int64_t)b * p.ldc + n0 + 4 * n);
    }
  };
  load(first);
  int good = -1;   // lane j: the state row of batch row i + j (i a multiple of 32), while the first states are under way
  for (int i = 0, b = first; b < rows; ++i, b += stride) {
    if (i % 32 == 0) good = state_slots_block(p.slots, b, stride, rows, p.n_slots, table, p.status);   // i is the block's
    const int here = __shfl_sync(0xffffffffu, good, i % 32);
    float x[4], Bn[NPL], Cn[NPL];
    Four<T>::unpack(rx, x);
#pragma unroll
    for (int n = 0; n < NPL / 4; ++n) {
      Four<T>::unpack(rB[n], reinterpret_cast<float(&)[4]>(Bn[4 * n]));
      Four<T>::unpack(rC[n], reinterpret_cast<float(&)[4]>(Cn[4 * n]));
    }
    const float delta = softplus_f(Elem<T>::to_f(rdt) + bias), z = Elem<T>::to_f(rz);
    load(b + stride);
    copies_wait<kStepDepth - 2>();
    fetch(i + kStepDepth - 1);
    if (here < 0 || !in_bounds(here < p.n_slots, p.status)) continue;
    float2 dl[2], dx[2], y[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      dl[k].x = __shfl_sync(0xffffffffu, delta, (lane & 7) + 16 * k);
      dl[k].y = __shfl_sync(0xffffffffu, delta, (lane & 7) + 16 * k + 8);
      dx[k] = mul2(dl[k], make_float2(x[2 * k], x[2 * k + 1]));
    }
    if (active) {
      float4* st = state_of(here);
      const float4* h4 = &ring[i % kStepDepth][0][threadIdx.x];
#pragma unroll
      for (int n = 0; n < NPL; ++n) {
        const float4 old = h4[n * kThreads];
        float2 h[2] = {make_float2(old.x, old.y), make_float2(old.z, old.w)};
        const float2 B2 = make_float2(Bn[n], Bn[n]), C2 = make_float2(Cn[n], Cn[n]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 e = mul2(dl[k], A[n][k]);
          h[k] = fma2(make_float2(ex2(e.x), ex2(e.y)), h[k], mul2(dx[k], B2));
          y[k] = fma2(C2, h[k], y[k]);
        }
        st[n * ld4] = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
      }
    }
    // sum over the four lanes of a channel group, halving the channels a lane holds: lane oc ends with channel oc
    const bool up2 = (oc & 2) != 0, up1 = (oc & 1) != 0;
    float2 s = up2 ? y[1] : y[0];
    const float2 give = up2 ? y[0] : y[1];
    s.x += __shfl_xor_sync(0xffffffffu, give.x, 16);
    s.y += __shfl_xor_sync(0xffffffffu, give.y, 16);
    float out = (up1 ? s.y : s.x) + __shfl_xor_sync(0xffffffffu, up1 ? s.x : s.y, 8);
    const float xo = oc == 0 ? x[0] : oc == 1 ? x[1] : oc == 2 ? x[2] : x[3];
    out = fmaf(skip, xo, out);
    if (p.z) out *= silu_f(z);
    if (active) store_elem(static_cast<T*>(p.y) + (int64_t)b * p.ldy + c0 + oc, out);
  }
}

// How a prompt batch is cut.  A variant is LPC lanes a channel (kThreads / LPC * CPT channels a block, `blocks`
// of them on an SM); the tiles are as many as make one wave of blocks, so that none waits for a second.
struct ScanPlan {
  int lpc, tile_len, tiles, groups;
};
constexpr int kSMs = 148;   // a B200's: the workspace's size follows from it, and is asked for without a device
constexpr int scan_cpt(int lpc, int NS) { return lpc <= 2 && NS == 16 ? 2 : 1; }
constexpr int scan_blocks(int lpc) { return lpc == 1 ? 3 : lpc == 2 ? 4 : 5; }

// One lane a channel costs the fewest instructions and is right where the SMs are full for long; two lanes halve the
// work of a lone warp and double the warps, right below 2^27 tokens x channels x states (B200, bf16, us with 1 / 2 /
// 4 lanes: 16384 x 1024 x 16 176 / 189 / 242, 8192 x 1024 x 16 97 / 100 / 124, 4096 x 1024 x 16 58 / 56 / 66,
// 2048 x 1024 x 16 37 / 32 / 36, 512 x 1024 x 16 19 / 15 / 14). Four lanes need 32 channels a block instead of 256 or
// 128: for a D that would leave most of a block idle.
// Up to kOneTile tokens, eight lanes a channel and a single tile, one launch instead of three (us, single against three:
// 17 x 1024 x 16 4.2 / 11.6, 61 tokens 6.9 / 11.6, 96 8.6 / 11.9, 190 15.3 / 12.2; 128 x 4096 x 16 12.9 / 18.2,
// 128 x 16384 x 16 29.6 / 38.3).
constexpr int kOneTile = 128, kMinTile = 16;
int scan_width(int lpc, int32_t N) { return kThreads / lpc * scan_cpt(lpc, N); }   // channels a block
int scan_groups(int lpc, int32_t D, int32_t N) { return (D + scan_width(lpc, N) - 1) / scan_width(lpc, N); }
int64_t scan_wave(int lpc, int32_t D, int32_t N) { return max(1, kSMs * scan_blocks(lpc) / scan_groups(lpc, D, N)); }

ScanPlan scan_plan(int64_t T, int32_t D, int32_t N) {
  ScanPlan p{8, kOneTile, 1, 0};
  if (T > kOneTile) {
    const bool large = T * D * N >= ((int64_t)1 << 27);
    const int lanes[3] = {1, 2, 4};
    const double cost[3] = {large ? 1.0 : 1.15, large ? 1.06 : 1.0, large ? 1.37 : 1.1};   // a full block's, measured
    double best = 0;
    for (int v = 0; v < 3; ++v) {
      const double c = cost[v] * scan_groups(lanes[v], D, N) * scan_width(lanes[v], N) / D;
      if (v == 0 || c < best) {
        best = c;
        p.lpc = lanes[v];
      }
    }
  }
  p.groups = scan_groups(p.lpc, D, N);
  if (T > kOneTile) {
    const int64_t tiles = scan_wave(p.lpc, D, N);
    p.tile_len = (int)max((T + tiles - 1) / tiles, (int64_t)kMinTile);
    p.tiles = (int)((T + p.tile_len - 1) / p.tile_len);
  }
  return p;
}

template <typename T, int NS, int LPC>
cudaError_t launch_tiles(const SelScanArgs& a, const ScanPlan& p, cudaStream_t s) {
  constexpr int CPT = scan_cpt(LPC, NS), MINB = scan_blocks(LPC);
  // state pairs whose decays run on the FMA pipe: one of 8 or two of 16 take 4% off (181 against 189 us, 319 against
  // 331); more cost more than they save (2 of 8: 188), and so does any with several lanes a channel
  constexpr int POLY = LPC == 1 ? NS / 16 : 0;
  const int64_t blocks = (int64_t)p.groups * p.tiles;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if constexpr (LPC != 8) {   // eight lanes: one tile always
    if (p.tiles > 1) {
      cudaError_t e = launch_dependent(scan_tile_kernel<T, CPT, LPC, NS, false, MINB, POLY>,
                                       dim3((unsigned)(blocks - p.groups)), kThreads, s, a, p.tile_len, p.tiles);
      if (e != cudaSuccess) return e;
      const int warps = min((p.tiles - 1 + kJoin - 1) / kJoin, kJoinWarps);
      e = launch_dependent(scan_join_kernel<NS>, dim3(NS * a.D / 32), 32 * warps, s, a, p.tiles);
      if (e != cudaSuccess) return e;
    }
  }
  return launch_dependent(scan_tile_kernel<T, CPT, LPC, NS, true, MINB, POLY>, dim3((unsigned)blocks), kThreads, s, a,
                          p.tile_len, p.tiles);
}

template <typename T, int NS>
cudaError_t launch_scan(const SelScanArgs& a, cudaStream_t s) {
  const ScanPlan p = scan_plan(a.T, a.D, NS);
  if (p.lpc == 1) return launch_tiles<T, NS, 1>(a, p, s);
  if (p.lpc == 2) return launch_tiles<T, NS, 2>(a, p, s);
  if (p.lpc == 4) return launch_tiles<T, NS, 4>(a, p, s);
  return launch_tiles<T, NS, 8>(a, p, s);
}

template <typename T, int NS>
cudaError_t launch_step(const SelScanArgs& a, cudaStream_t s) {
  const int64_t groups = (a.D + kThreads - 1) / kThreads;
  // one wave of blocks, each with the same number of batch rows but for the last
  const int64_t wave = max((int64_t)1, kSMs * step_blocks(NS) / groups);
  const int64_t each = (a.T + wave - 1) / wave;
  const int64_t blocks = groups * ((a.T + each - 1) / each);
  return launch_dependent(scan_step_kernel<T, NS>, dim3((unsigned)blocks), kThreads, s, a, (int)groups);
}
}  // namespace

// The most tiles that any variant cuts T rows or fewer into: it grows with T, so a workspace for the largest call
// serves every smaller one.
size_t selective_scan_workspace_bytes(int64_t T, int32_t D, int32_t N) {
  if (T <= kOneTile) return 0;
  int64_t tiles = 1;
  for (int lpc = 1; lpc <= 4; lpc *= 2) tiles = max(tiles, min(scan_wave(lpc, D, N), (T + kMinTile - 1) / kMinTile));
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
