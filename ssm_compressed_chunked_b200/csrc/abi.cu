// extern "C" entry points: host-side validation, then the stream-ordered launches.
// The passages each entry point follows are cited in include/attamba.h.
#include <stdio.h>
#include <string.h>

#include "attamba.h"
#include "launch.h"

namespace {
thread_local char g_err[256] = "";

attamba_status_t cuda_fail(cudaError_t e, const char* where) {
  snprintf(g_err, sizeof(g_err), "%s: %s", where, cudaGetErrorString(e));
  return ATTAMBA_ERR_CUDA;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_dtype(attamba_dtype_t d) { return d == ATTAMBA_F32 || d == ATTAMBA_BF16; }
constexpr int64_t kMaxTokens = (int64_t)1 << 31;
}  // namespace

extern "C" {

const char* attamba_version(void) {
#if defined(ATTAMBA_CHECKED)
  return "attamba-b200 0.1 (sm_100a) checked";
#else
  return "attamba-b200 0.1 (sm_100a)";
#endif
}

const char* attamba_status_string(attamba_status_t s) {
  switch (s) {
    case ATTAMBA_OK: return "ok";
    case ATTAMBA_ERR_INVALID_ARG: return "invalid argument";
    case ATTAMBA_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case ATTAMBA_ERR_CUDA: return "CUDA error";
  }
  return "unknown status";
}

const char* attamba_last_error(void) { return g_err; }

int32_t attamba_uniform_chunk_count(int32_t n, int32_t P, int32_t offset) {
  if (n < 1 || P < 1) return -1;
  const int32_t o = ((offset % P) + P) % P;
  // starts: 0, then o + kP in (0, n)
  int32_t cnt = 1;
  const int32_t first = (o == 0) ? P : o;
  if (first < n) cnt += 1 + (n - 1 - first) / P;
  return cnt;
}

attamba_status_t attamba_chunk_index(const int32_t* cu_in, int32_t n_chunks, int32_t B, int32_t n,
                                     int32_t P, int32_t offset, int32_t L, attamba_mask_t mode,
                                     const attamba_index_t* out, int32_t* d_status,
                                     attamba_stream_t stream) {
  if (!out || B < 1 || n < 1 || (int64_t)B * n >= kMaxTokens || L < 0 || n_chunks < B)
    return ATTAMBA_ERR_INVALID_ARG;
  if (mode != ATTAMBA_MASK_TRAIN && mode != ATTAMBA_MASK_TEST) return ATTAMBA_ERR_INVALID_ARG;
  if (!out->cu || !out->bpos || !out->bptr || !out->ls || !out->nbb) return ATTAMBA_ERR_INVALID_ARG;
  if (out->n_chunks != n_chunks || out->B != B || out->n != n) return ATTAMBA_ERR_INVALID_ARG;
  if (n_chunks > (int64_t)B * n) return ATTAMBA_ERR_INVALID_ARG;
  if (cu_in == nullptr) {
    if (P < 1) return ATTAMBA_ERR_INVALID_ARG;
    if ((int64_t)attamba_uniform_chunk_count(n, P, offset) * B != n_chunks) return ATTAMBA_ERR_INVALID_ARG;
  }
  cudaError_t e = attamba::launch_chunk_index(cu_in, n_chunks, B, n, P, offset, L, (int)mode, *out, d_status,
                                              reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_chunk_index");
}

namespace {
attamba_status_t scan_entry(attamba_dtype_t dtype, const void* u_k, const void* u_v, const void* dt_k,
                            const void* dt_v, const float* bias_k, const float* bias_v, const float* A_k,
                            const float* A_v, const void* B_k, const void* C_k, const void* B_v, const void* C_v,
                            const int32_t* cu, int32_t n_chunks, int64_t T, int32_t D, int32_t N, void* K,
                            void* V, void* Kc, void* Vc, int32_t* d_status, cudaStream_t stream, const char* name) {
  if (!ok_dtype(dtype)) return ATTAMBA_ERR_UNSUPPORTED;
  if (N != 16 && N != 32) return ATTAMBA_ERR_UNSUPPORTED;
  if (T < 1 || T >= kMaxTokens || D < 8 || D % 8 != 0 || n_chunks < 1 || n_chunks > T)
    return ATTAMBA_ERR_INVALID_ARG;
  const void* req[] = {u_k, u_v, dt_k, dt_v, bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, cu, K, V};
  for (const void* p : req)
    if (!p || !aligned16(p)) return ATTAMBA_ERR_INVALID_ARG;
  if ((Kc == nullptr) != (Vc == nullptr)) return ATTAMBA_ERR_INVALID_ARG;
  if (Kc && (!aligned16(Kc) || !aligned16(Vc))) return ATTAMBA_ERR_INVALID_ARG;
  attamba::ScanArgs a{};
  a.x[0] = u_k; a.x[1] = u_v;
  a.dt[0] = dt_k; a.dt[1] = dt_v;
  a.bias[0] = bias_k; a.bias[1] = bias_v;
  a.A[0] = A_k; a.A[1] = A_v;
  a.Bm[0] = B_k; a.Bm[1] = B_v;
  a.Cm[0] = C_k; a.Cm[1] = C_v;
  a.cu = cu;
  a.n_chunks = n_chunks;
  a.T = T;
  a.D = D;
  a.N = N;
  a.out[0] = K; a.out[1] = V;
  a.outc[0] = Kc; a.outc[1] = Vc;
  a.status = d_status;
  cudaError_t e = attamba::launch_kv_ssm_scan(dtype, a, stream);
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, name);
}
}  // namespace

attamba_status_t attamba_kv_ssm_scan(attamba_dtype_t dtype, const void* x, const void* dt_k,
                                     const void* dt_v, const float* bias_k, const float* bias_v,
                                     const float* A_k, const float* A_v, const void* B_k,
                                     const void* C_k, const void* B_v, const void* C_v,
                                     const int32_t* cu, int32_t n_chunks, int64_t T, int32_t D,
                                     int32_t N, void* K, void* V, void* Kc, void* Vc,
                                     int32_t* d_status, attamba_stream_t stream) {
  return scan_entry(dtype, x, x, dt_k, dt_v, bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, cu, n_chunks, T, D, N,
                    K, V, Kc, Vc, d_status, reinterpret_cast<cudaStream_t>(stream), "attamba_kv_ssm_scan");
}

attamba_status_t attamba_kv_ssm_scan_u(attamba_dtype_t dtype, const void* u_k, const void* u_v,
                                       const void* dt_k, const void* dt_v, const float* bias_k,
                                       const float* bias_v, const float* A_k, const float* A_v,
                                       const void* B_k, const void* C_k, const void* B_v, const void* C_v,
                                       const int32_t* cu, int32_t n_chunks, int64_t T, int32_t D, int32_t N,
                                       void* K, void* V, void* Kc, void* Vc, int32_t* d_status,
                                       attamba_stream_t stream) {
  return scan_entry(dtype, u_k, u_v, dt_k, dt_v, bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, cu, n_chunks, T, D,
                    N, K, V, Kc, Vc, d_status, reinterpret_cast<cudaStream_t>(stream), "attamba_kv_ssm_scan_u");
}

attamba_status_t attamba_proj_gemm(attamba_dtype_t dtype, const void* X, const void* W, int64_t M, int32_t Nout,
                                   int32_t K, const attamba_proj_seg_t* segs, int32_t nseg, int32_t* d_status,
                                   attamba_stream_t stream) {
  if (dtype != ATTAMBA_BF16) return ATTAMBA_ERR_UNSUPPORTED;
  if (M < 1 || Nout < 1 || K < 64 || K % 64 != 0 || !segs || nseg < 1 || nseg > attamba::kMaxProjSegs)
    return ATTAMBA_ERR_INVALID_ARG;
  if (M >= ((int64_t)1 << 31) || M * (int64_t)K >= ((int64_t)1 << 40) || M * (int64_t)Nout >= ((int64_t)1 << 40))
    return ATTAMBA_ERR_INVALID_ARG;
  if (!X || !W || !aligned16(X) || !aligned16(W)) return ATTAMBA_ERR_INVALID_ARG;
  attamba::ProjArgs a{};
  a.X = X; a.W = W; a.M = M; a.Nout = Nout; a.K = K; a.nseg = nseg; a.status = d_status;
  int32_t end = 0;
  for (int s = 0; s < nseg; ++s) {
    const attamba_proj_seg_t& g = segs[s];
    if (!g.ptr || !aligned16(g.ptr) || g.col0 < end || g.width < 8 || g.col0 % 8 != 0 || g.width % 8 != 0 ||
        (int64_t)g.col0 + g.width > Nout)
      return ATTAMBA_ERR_INVALID_ARG;
    a.seg_ptr[s] = g.ptr;
    a.seg_col0[s] = g.col0;
    a.seg_width[s] = g.width;
    end = g.col0 + g.width;
  }
  cudaError_t e = attamba::launch_proj_gemm(a, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return ATTAMBA_ERR_UNSUPPORTED;
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_proj_gemm");
}

attamba_status_t attamba_chunk_attn_fwd(attamba_dtype_t dtype, const void* q, const void* K,
                                        const void* V, const void* Kc, const void* Vc,
                                        const attamba_index_t* idx, int32_t H, int32_t dh,
                                        float scale, void* O, float* lse, int32_t* d_status,
                                        attamba_stream_t stream) {
  if (!ok_dtype(dtype)) return ATTAMBA_ERR_UNSUPPORTED;
  if (dh != 64) return ATTAMBA_ERR_UNSUPPORTED;
  if (!idx || H < 1 || idx->B < 1 || idx->n < 1 || idx->n_chunks < idx->B) return ATTAMBA_ERR_INVALID_ARG;
  const int64_t T = (int64_t)idx->B * idx->n;
  if (T >= kMaxTokens || T * H >= kMaxTokens) return ATTAMBA_ERR_INVALID_ARG;
  const void* req[] = {q, K, V, Kc, Vc, O};
  for (const void* p : req)
    if (!p || !aligned16(p)) return ATTAMBA_ERR_INVALID_ARG;
  if (!idx->bpos || !idx->bptr || !idx->ls || !idx->nbb) return ATTAMBA_ERR_INVALID_ARG;
  if (!(scale > 0.f)) return ATTAMBA_ERR_INVALID_ARG;
  attamba::AttnArgs a{};
  a.q = q; a.K = K; a.V = V; a.Kc = Kc; a.Vc = Vc;
  a.bpos = idx->bpos; a.bptr = idx->bptr; a.ls = idx->ls; a.nbb = idx->nbb;
  a.B = idx->B; a.n = idx->n; a.H = H; a.dh = dh; a.n_chunks = idx->n_chunks;
  a.scale = scale; a.O = O; a.lse = lse; a.status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = (dtype == ATTAMBA_BF16) ? attamba::launch_chunk_attn_bf16(a, s) : attamba::launch_chunk_attn_f32(a, s);
  if (e == cudaErrorNotSupported) {
    snprintf(g_err, sizeof(g_err), "attamba_chunk_attn_fwd: cuTensorMapEncodeTiled unavailable or rejected");
    return ATTAMBA_ERR_CUDA;
  }
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_chunk_attn_fwd");
}

attamba_status_t attamba_selftest_wait_timeout(uint64_t limit_ns, int32_t* d_status, attamba_stream_t stream) {
  if (!d_status || limit_ns < 1000 || limit_ns > 1000000000ull) return ATTAMBA_ERR_INVALID_ARG;
  const cudaError_t e = attamba::launch_wait_selftest(limit_ns, d_status, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_selftest_wait_timeout");
}

size_t attamba_cache_bytes(const attamba_cache_t* cache) {
  if (!cache || cache->B < 1 || cache->H < 1 || cache->N < 1 || cache->L < 1 || cache->cap < 1 || cache->dh != 64)
    return 0;
  const uint64_t B = (uint64_t)cache->B, H = (uint64_t)cache->H, dh = (uint64_t)cache->dh;
  const uint64_t N = (uint64_t)cache->N, L = (uint64_t)cache->L, cap = (uint64_t)cache->cap;
  auto up = [](uint64_t bytes) { return (bytes + 255) & ~uint64_t(255); };
  const uint64_t bytes = up(2 * B * N * H * dh * 4)          // state [2, B, N, D] fp32
                         + 2 * up(B * H * cap * dh * 2)     // Kb, Vb [B, H, cap, dh] bf16
                         + up(B * cap * 4)                  // bpos [B, cap] int32
                         + 2 * up(B * H * L * dh * 2)       // Kr, Vr [B, H, L, dh] bf16
                         + 2 * up(B * 4);                   // nb, pos [B] int32
  return (size_t)bytes;
}

size_t attamba_decode_workspace_size(const attamba_cache_t* cache) {
  if (!cache || cache->B < 1 || cache->H < 1 || cache->cap < 1 || cache->L < 1) return 0;
  return attamba::decode_workspace_bytes(*cache);
}

attamba_status_t attamba_decode_step(attamba_dtype_t dtype, const attamba_cache_t* cache,
                                     const void* q_t, const void* x_t, const void* dt_k,
                                     const void* dt_v, const float* bias_k, const float* bias_v,
                                     const float* A_k, const float* A_v, const void* B_k,
                                     const void* C_k, const void* B_v, const void* C_v,
                                     float scale, void* o_t, void* workspace,
                                     size_t workspace_bytes, int32_t* d_status,
                                     attamba_stream_t stream) {
  if (dtype != ATTAMBA_BF16) return ATTAMBA_ERR_UNSUPPORTED;
  if (!cache) return ATTAMBA_ERR_INVALID_ARG;
  const attamba_cache_t& c = *cache;
  if (c.dh != 64 || (c.N != 16 && c.N != 32)) return ATTAMBA_ERR_UNSUPPORTED;
  if (c.B < 1 || c.H < 1 || c.P < 1 || c.L < 1 || c.cap < 1) return ATTAMBA_ERR_INVALID_ARG;
  if ((int64_t)c.B * c.H * c.cap * c.dh >= ((int64_t)1 << 40)) return ATTAMBA_ERR_INVALID_ARG;
  const void* req[] = {c.state, c.Kb, c.Vb, c.bpos, c.Kr, c.Vr, c.nb, c.pos, q_t, x_t, dt_k, dt_v,
                       bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, o_t, workspace};
  for (const void* p : req)
    if (!p) return ATTAMBA_ERR_INVALID_ARG;
  const void* al[] = {c.Kb, c.Vb, c.Kr, c.Vr, q_t, workspace};
  for (const void* p : al)
    if (!aligned16(p)) return ATTAMBA_ERR_INVALID_ARG;
  if (workspace_bytes < attamba::decode_workspace_bytes(c)) return ATTAMBA_ERR_INVALID_ARG;
  if (!(scale > 0.f)) return ATTAMBA_ERR_INVALID_ARG;
  attamba::DecodeArgs a{};
  a.c = c;
  a.q = q_t; a.x = x_t;
  a.dt[0] = dt_k; a.dt[1] = dt_v;
  a.bias[0] = bias_k; a.bias[1] = bias_v;
  a.A[0] = A_k; a.A[1] = A_v;
  a.Bm[0] = B_k; a.Bm[1] = B_v;
  a.Cm[0] = C_k; a.Cm[1] = C_v;
  a.scale = scale; a.o = o_t;
  a.work = static_cast<float*>(workspace);
  a.splits = attamba::decode_splits(c);
  a.status = d_status;
  cudaError_t e = attamba::launch_decode_step(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_decode_step");
}

attamba_status_t attamba_cache_from_prefill(attamba_dtype_t dtype, const attamba_cache_t* cache,
                                            const void* K, const void* V, const void* x,
                                            const void* dt_k, const void* dt_v, const float* bias_k,
                                            const float* bias_v, const float* A_k, const float* A_v,
                                            const void* B_k, const void* C_k, const void* B_v,
                                            const void* C_v, int32_t n0, int32_t* d_status,
                                            attamba_stream_t stream) {
  (void)d_status;  // nothing is detected on the device: every limit is checked here
  if (dtype != ATTAMBA_BF16) return ATTAMBA_ERR_UNSUPPORTED;
  if (!cache) return ATTAMBA_ERR_INVALID_ARG;
  const attamba_cache_t& c = *cache;
  if (c.dh != 64 || (c.N != 16 && c.N != 32)) return ATTAMBA_ERR_UNSUPPORTED;
  if (c.B < 1 || c.H < 1 || c.P < 1 || c.L < 1 || c.cap < 1 || n0 < 1) return ATTAMBA_ERR_INVALID_ARG;
  if ((int64_t)c.B * c.H * c.cap * c.dh >= ((int64_t)1 << 40)) return ATTAMBA_ERR_INVALID_ARG;
  if ((int64_t)c.B * n0 * c.H * c.dh >= ((int64_t)1 << 40)) return ATTAMBA_ERR_INVALID_ARG;
  const void* req[] = {c.state, c.Kb, c.Vb, c.bpos, c.Kr, c.Vr, c.nb, c.pos, K, V, x, dt_k, dt_v,
                       bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v};
  for (const void* p : req)
    if (!p) return ATTAMBA_ERR_INVALID_ARG;
  const void* al[] = {c.Kb, c.Vb, c.Kr, c.Vr, K, V};
  for (const void* p : al)
    if (!aligned16(p)) return ATTAMBA_ERR_INVALID_ARG;
  const int32_t nb = attamba::handoff_boundaries(n0, c.P, c.offset);
  if (nb > c.cap) {
    snprintf(g_err, sizeof(g_err), "attamba_cache_from_prefill: %d boundaries in [0, %d) exceed cap %d", nb, n0,
             c.cap);
    return ATTAMBA_ERR_INVALID_ARG;
  }
  attamba::HandoffArgs a{};
  a.c = c;
  a.K = K; a.V = V; a.x = x;
  a.dt[0] = dt_k; a.dt[1] = dt_v;
  a.bias[0] = bias_k; a.bias[1] = bias_v;
  a.A[0] = A_k; a.A[1] = A_v;
  a.Bm[0] = B_k; a.Bm[1] = B_v;
  a.Cm[0] = C_k; a.Cm[1] = C_v;
  a.n0 = n0;
  a.nb = nb;
  cudaError_t e = attamba::launch_cache_from_prefill(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_cache_from_prefill");
}

attamba_status_t attamba_decode_step_noalloc(attamba_dtype_t dtype, const attamba_cache_t* cache,
                                             const void* q_t, const void* x_t, const void* dt_k,
                                             const void* dt_v, const float* bias_k, const float* bias_v,
                                             const float* A_k, const float* A_v, const void* B_k,
                                             const void* C_k, const void* B_v, const void* C_v,
                                             float scale, void* o_t, int32_t* d_status,
                                             attamba_stream_t stream) {
  if (dtype != ATTAMBA_BF16) return ATTAMBA_ERR_UNSUPPORTED;
  if (!cache) return ATTAMBA_ERR_INVALID_ARG;
  const attamba_cache_t& c = *cache;
  if (c.dh != 64 || (c.N != 16 && c.N != 32)) return ATTAMBA_ERR_UNSUPPORTED;
  if (c.B < 1 || c.H < 1 || c.P < 1 || c.L < 1 || c.cap < 1) return ATTAMBA_ERR_INVALID_ARG;
  if ((int64_t)c.B * c.H * c.cap * c.dh >= ((int64_t)1 << 40)) return ATTAMBA_ERR_INVALID_ARG;
  const void* req[] = {c.state, c.Kb, c.Vb, c.bpos, c.Kr, c.Vr, c.nb, c.pos, q_t, x_t, dt_k, dt_v,
                       bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, o_t};
  for (const void* p : req)
    if (!p) return ATTAMBA_ERR_INVALID_ARG;
  const void* al[] = {c.Kb, c.Vb, c.Kr, c.Vr, q_t};
  for (const void* p : al)
    if (!aligned16(p)) return ATTAMBA_ERR_INVALID_ARG;
  if (!(scale > 0.f)) return ATTAMBA_ERR_INVALID_ARG;
  const size_t need = attamba::decode_workspace_bytes(c);
  if (need > attamba::decode_noalloc_scratch_bytes()) {
    snprintf(g_err, sizeof(g_err),
             "attamba_decode_step_noalloc: this cache needs %zu bytes of split-K scratch, the built-in "
             "scratch holds %zu; use attamba_decode_step with a workspace",
             need, attamba::decode_noalloc_scratch_bytes());
    return ATTAMBA_ERR_UNSUPPORTED;
  }
  float* scratch = nullptr;
  cudaError_t e = attamba::decode_noalloc_scratch(&scratch);
  if (e != cudaSuccess) return cuda_fail(e, "attamba_decode_step_noalloc (scratch address)");
  attamba::DecodeArgs a{};
  a.c = c;
  a.q = q_t; a.x = x_t;
  a.dt[0] = dt_k; a.dt[1] = dt_v;
  a.bias[0] = bias_k; a.bias[1] = bias_v;
  a.A[0] = A_k; a.A[1] = A_v;
  a.Bm[0] = B_k; a.Bm[1] = B_v;
  a.Cm[0] = C_k; a.Cm[1] = C_v;
  a.scale = scale; a.o = o_t;
  a.work = scratch;
  a.splits = attamba::decode_splits(c);
  a.status = d_status;
  e = attamba::launch_decode_step(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_decode_step_noalloc");
}

namespace {
// A refusal with its reason as the thread's error text.
attamba_status_t refuse(attamba_status_t st, const char* what, const char* why) {
  snprintf(g_err, sizeof(g_err), "%s: %s", what, why);
  return st;
}
constexpr attamba_status_t kInvalid = ATTAMBA_ERR_INVALID_ARG, kUnsupported = ATTAMBA_ERR_UNSUPPORTED;

// Token rows an operator of the SSM block reads or writes: rows x cols elements of `es` bytes, `ld` apart.
struct Rows {
  const void* p;
  int64_t rows, ld;
  int32_t cols;
  int es;
  bool out;
  const char* name;
};
bool ok_rows(const Rows& r) {
  return aligned16(r.p) && r.ld >= r.cols && r.ld < ((int64_t)1 << 31) && (r.ld * r.es) % 16 == 0 &&
         r.rows <= ((int64_t)1 << 56) / (r.ld * r.es);
}
// whether two row sets share a byte: column windows of one wide array (same stride) do not
bool overlap(const Rows& a, const Rows& b) {
  const int64_t as = a.ld * a.es, bs = b.ld * b.es, ac = (int64_t)a.cols * a.es, bc = (int64_t)b.cols * b.es;
  const intptr_t pa = reinterpret_cast<intptr_t>(a.p), pb = reinterpret_cast<intptr_t>(b.p);
  const intptr_t ea = pa + (a.rows - 1) * as + ac, eb = pb + (b.rows - 1) * bs + bc;
  if (ea <= pb || eb <= pa) return false;
  if (as != bs) return true;
  const int64_t off = (((pb - pa) % as) + as) % as;   // b's window starts `off` bytes into a's row
  return off < ac || off + bc > as;
}
// every given row set is well formed and no output shares memory with another set
attamba_status_t check_rows(const Rows* r, int n, const char* what) {
  for (int i = 0; i < n; ++i) {
    if (!r[i].p) continue;
    if (!ok_rows(r[i])) {
      snprintf(g_err, sizeof(g_err), "%s: %s must be 16-byte aligned with a row stride of a multiple of 16 bytes", what,
               r[i].name);
      return ATTAMBA_ERR_INVALID_ARG;
    }
    for (int j = 0; j < n; ++j)
      if (j != i && r[i].out && r[j].p && overlap(r[i], r[j])) {
        snprintf(g_err, sizeof(g_err), "%s: %s overlaps %s", what, r[i].name, r[j].name);
        return ATTAMBA_ERR_INVALID_ARG;
      }
  }
  return ATTAMBA_OK;
}
int elem_size(attamba_dtype_t d) { return d == ATTAMBA_BF16 ? 2 : 4; }
constexpr int64_t kMaxSeqTokens = ((int64_t)1 << 31) - 65536;   // token positions plus a tile stay int32
constexpr int32_t kMaxChannels = 1 << 20;
constexpr int32_t kMaxRows = 1 << 20;                           // sequences or batch rows of one call
// with a slot map: every row's slot is looked for among the ones ahead of it, which grows with the square: at 8192 rows it
// takes a quarter of a decode step (D 1024, N 16: 234 us, 180 without a map), and most of a prompt batch of that many
constexpr int32_t kMaxSlots = 8192;
bool too_many(const int32_t* slots, int32_t rows, const char* what) {
  if (rows <= (slots ? kMaxSlots : kMaxRows)) return false;
  snprintf(g_err, sizeof(g_err), "%s: %d sequences in one call, at most %d%s", what, rows, slots ? kMaxSlots : kMaxRows,
           slots ? " with slots" : "");
  return true;
}
bool ok_channels(int32_t D) { return D >= 8 && D % 8 == 0 && D <= kMaxChannels; }
bool ok_seqs(const attamba_seqs_t* q) {
  return q && q->cu && q->T >= 1 && q->T < kMaxSeqTokens && q->S >= 1;
}

attamba_status_t conv_entry(attamba_dtype_t dtype, attamba::ConvArgs& a, int64_t ldx, int64_t ldy, int32_t K,
                            attamba_act_t act, bool step, cudaStream_t s, const char* name) {
  if (!ok_dtype(dtype)) return refuse(kUnsupported, name, "dtype is F32 or BF16");
  if (K < 2 || K > 4) return refuse(kUnsupported, name, "K is 2, 3 or 4");
  if (!a.x || !a.w || !a.y) return refuse(kInvalid, name, "x, w and y are required");
  if (!ok_channels(a.D)) return refuse(kInvalid, name, "D is a multiple of 8, at most 2^20");
  if (act != ATTAMBA_ACT_LINEAR && act != ATTAMBA_ACT_SILU) return refuse(kInvalid, name, "act is LINEAR or SILU");
  if (a.state && a.n_slots < 1) return refuse(kInvalid, name, "a state has at least one slot");
  if (!aligned16(a.w) || !aligned16(a.bias) || !aligned16(a.state))
    return refuse(kInvalid, name, "w, bias and state are 16-byte aligned");
  const int es = elem_size(dtype);
  const Rows rows[] = {{a.x, a.T, ldx, a.D, es, false, "x"},
                       {a.y, a.T, ldy, a.D, es, true, "y"},
                       {a.state, (int64_t)a.n_slots * (K - 1), a.D, a.D, es, true, "state"}};
  const attamba_status_t st = check_rows(rows, 3, name);
  if (st != ATTAMBA_OK) return st;
  a.ldx = (int32_t)ldx;
  a.ldy = (int32_t)ldy;
  a.act = (int32_t)act;
  const cudaError_t e = step ? attamba::launch_conv_step(dtype, K, a, s) : attamba::launch_causal_conv(dtype, K, a, s);
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, name);
}

attamba_status_t check_scan(attamba_dtype_t dtype, attamba::SelScanArgs& a, int64_t ldx, int64_t lddt, int64_t ldb,
                            int64_t ldc, int64_t ldz, int64_t ldy, const char* name) {
  if (!ok_dtype(dtype)) return refuse(kUnsupported, name, "dtype is F32 or BF16");
  if (a.N != 16 && a.N != 32) return refuse(kUnsupported, name, "N is 16 or 32");
  if (!a.x || !a.dt || !a.A || !a.Bm || !a.Cm || !a.y) return refuse(kInvalid, name, "x, dt, A, B, C and y are required");
  if (!ok_channels(a.D)) return refuse(kInvalid, name, "D is a multiple of 8, at most 2^20");
  if (a.state && a.n_slots < 1) return refuse(kInvalid, name, "a state has at least one slot");
  if (!aligned16(a.A) || !aligned16(a.bias) || !aligned16(a.skip))
    return refuse(kInvalid, name, "A, bias and skip are 16-byte aligned");
  const int es = elem_size(dtype);
  const Rows rows[] = {{a.x, a.T, ldx, a.D, es, false, "x"},   {a.dt, a.T, lddt, a.D, es, false, "dt"},
                       {a.Bm, a.T, ldb, a.N, es, false, "B"},  {a.Cm, a.T, ldc, a.N, es, false, "C"},
                       {a.z, a.T, ldz, a.D, es, false, "z"},   {a.y, a.T, ldy, a.D, es, true, "y"},
                       {a.state, (int64_t)a.n_slots * a.N, a.D, a.D, 4, true, "state"}};
  const attamba_status_t st = check_rows(rows, 7, name);
  if (st != ATTAMBA_OK) return st;
  a.ldx = (int32_t)ldx;
  a.lddt = (int32_t)lddt;
  a.ldb = (int32_t)ldb;
  a.ldc = (int32_t)ldc;
  a.ldz = (int32_t)ldz;
  a.ldy = (int32_t)ldy;
  return ATTAMBA_OK;
}
}  // namespace

attamba_status_t attamba_causal_conv(attamba_dtype_t dtype, const void* x, int64_t ldx, const float* w,
                                     const float* bias, int32_t D, int32_t K, attamba_act_t act,
                                     const attamba_seqs_t* seqs, void* state, int32_t n_slots, void* y,
                                     int64_t ldy, int32_t* d_status, attamba_stream_t stream) {
  if (!ok_seqs(seqs)) return refuse(kInvalid, "attamba_causal_conv", "a sequence table has cu, S >= 1 and 1 <= T < 2^31 - 65536");
  if (too_many(seqs->slots, seqs->S, "attamba_causal_conv")) return ATTAMBA_ERR_UNSUPPORTED;
  attamba::ConvArgs a{};
  a.x = x; a.w = w; a.bias = bias; a.state = state; a.y = y;
  a.cu = seqs->cu; a.slots = seqs->slots; a.cont = seqs->cont;
  a.T = seqs->T; a.S = seqs->S; a.D = D; a.n_slots = n_slots; a.status = d_status;
  return conv_entry(dtype, a, ldx, ldy, K, act, false, reinterpret_cast<cudaStream_t>(stream), "attamba_causal_conv");
}

attamba_status_t attamba_conv_step(attamba_dtype_t dtype, const void* x, int64_t ldx, const float* w,
                                   const float* bias, int32_t D, int32_t K, attamba_act_t act, int32_t B,
                                   const int32_t* slots, void* state, int32_t n_slots, void* y, int64_t ldy,
                                   int32_t* d_status, attamba_stream_t stream) {
  if (B < 1 || !state) return refuse(kInvalid, "attamba_conv_step", "B >= 1 and a state are required");
  if (too_many(slots, B, "attamba_conv_step")) return ATTAMBA_ERR_UNSUPPORTED;
  attamba::ConvArgs a{};
  a.x = x; a.w = w; a.bias = bias; a.state = state; a.y = y; a.slots = slots;
  a.T = B; a.D = D; a.n_slots = n_slots; a.status = d_status;
  return conv_entry(dtype, a, ldx, ldy, K, act, true, reinterpret_cast<cudaStream_t>(stream), "attamba_conv_step");
}

size_t attamba_selective_scan_workspace_size(int64_t T, int32_t D, int32_t N) {
  if (T < 1 || T >= kMaxSeqTokens || !ok_channels(D) || (N != 16 && N != 32)) return 0;
  return attamba::selective_scan_workspace_bytes(T, D, N);
}

attamba_status_t attamba_selective_scan(attamba_dtype_t dtype, const void* x, int64_t ldx, const void* dt,
                                        int64_t lddt, const float* bias, const float* A, const void* B,
                                        int64_t ldb, const void* C, int64_t ldc, const float* skip, const void* z,
                                        int64_t ldz, int32_t D, int32_t N, const attamba_seqs_t* seqs, float* state,
                                        int32_t n_slots, void* y, int64_t ldy, void* workspace,
                                        size_t workspace_bytes, int32_t* d_status, attamba_stream_t stream) {
  if (!ok_seqs(seqs)) return refuse(kInvalid, "attamba_selective_scan", "a sequence table has cu, S >= 1 and 1 <= T < 2^31 - 65536");
  if (too_many(seqs->slots, seqs->S, "attamba_selective_scan")) return ATTAMBA_ERR_UNSUPPORTED;
  attamba::SelScanArgs a{};
  a.x = x; a.dt = dt; a.Bm = B; a.Cm = C; a.z = z; a.bias = bias; a.A = A; a.skip = skip; a.state = state; a.y = y;
  a.cu = seqs->cu; a.slots = seqs->slots; a.cont = seqs->cont;
  a.T = seqs->T; a.S = seqs->S; a.D = D; a.N = N; a.n_slots = n_slots;
  a.work = static_cast<float*>(workspace);
  a.status = d_status;
  const attamba_status_t st = check_scan(dtype, a, ldx, lddt, ldb, ldc, ldz, ldy, "attamba_selective_scan");
  if (st != ATTAMBA_OK) return st;
  const size_t need = attamba::selective_scan_workspace_bytes(a.T, D, N);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) {
    snprintf(g_err, sizeof(g_err), "attamba_selective_scan: needs %zu bytes of workspace, 16-byte aligned", need);
    return ATTAMBA_ERR_INVALID_ARG;
  }
  const cudaError_t e = attamba::launch_selective_scan(dtype, a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_selective_scan");
}

attamba_status_t attamba_scan_step(attamba_dtype_t dtype, const void* x, int64_t ldx, const void* dt, int64_t lddt,
                                   const float* bias, const float* A, const void* B, int64_t ldb, const void* C,
                                   int64_t ldc, const float* skip, const void* z, int64_t ldz, int32_t D, int32_t N,
                                   int32_t rows, const int32_t* slots, float* state, int32_t n_slots, void* y,
                                   int64_t ldy, int32_t* d_status, attamba_stream_t stream) {
  if (rows < 1 || !state) return refuse(kInvalid, "attamba_scan_step", "rows >= 1 and a state are required");
  if (too_many(slots, rows, "attamba_scan_step")) return ATTAMBA_ERR_UNSUPPORTED;
  attamba::SelScanArgs a{};
  a.x = x; a.dt = dt; a.Bm = B; a.Cm = C; a.z = z; a.bias = bias; a.A = A; a.skip = skip; a.state = state; a.y = y;
  a.slots = slots;
  a.T = rows; a.D = D; a.N = N; a.n_slots = n_slots; a.status = d_status;
  const attamba_status_t st = check_scan(dtype, a, ldx, lddt, ldb, ldc, ldz, ldy, "attamba_scan_step");
  if (st != ATTAMBA_OK) return st;
  const cudaError_t e = attamba::launch_scan_step(dtype, a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, "attamba_scan_step");
}

attamba_status_t attamba_clear_rows(attamba_dtype_t dtype, void* y, int64_t ldy, int32_t D, const attamba_seqs_t* seqs,
                                    int32_t B, const int32_t* slots, attamba_stream_t stream) {
  const char* name = "attamba_clear_rows";
  if (!ok_dtype(dtype)) return refuse(kUnsupported, name, "dtype is F32 or BF16");
  if (!y) return refuse(kInvalid, name, "y is required");
  if (!ok_channels(D)) return refuse(kInvalid, name, "D is a multiple of 8, at most 2^20");
  if ((seqs != nullptr) == (slots != nullptr)) return refuse(kInvalid, name, "a sequence table or slots, one of the two");
  if (seqs && !ok_seqs(seqs)) return refuse(kInvalid, name, "a sequence table has cu, S >= 1 and 1 <= T < 2^31 - 65536");
  if (seqs ? too_many(nullptr, seqs->S, name) : too_many(nullptr, B, name)) return ATTAMBA_ERR_UNSUPPORTED;
  if (!seqs && B < 1) return refuse(kInvalid, name, "B >= 1");
  const int es = elem_size(dtype);
  const Rows rows[] = {{y, seqs ? seqs->T : B, ldy, D, es, true, "y"}};
  const attamba_status_t st = check_rows(rows, 1, name);
  if (st != ATTAMBA_OK) return st;
  const cudaError_t e = attamba::launch_clear_rows(y, ldy * es, D * es, rows[0].rows, seqs ? seqs->cu + seqs->S : nullptr,
                                                   slots, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, name);
}

attamba_status_t attamba_block_norm(attamba_dtype_t dtype, attamba_dtype_t res_dtype, const void* y, int64_t ldy,
                                    const void* gate, int64_t ldg, attamba_act_t act, int32_t gate_first,
                                    const float* w_post, const void* res, int64_t ldr, const float* scale,
                                    float alpha, const float* w_pre, float eps, int64_t M, int32_t D, void* res_out,
                                    int64_t ldro, void* h, int64_t ldh, attamba_stream_t stream) {
  const char* name = "attamba_block_norm";
  if (!ok_dtype(dtype) || !ok_dtype(res_dtype)) return refuse(kUnsupported, name, "dtype and res_dtype are F32 or BF16");
  if (D < 8 || D % 8 != 0 || M < 1 || M > 0x7fffffff) return refuse(kInvalid, name, "D is a multiple of 8, 1 <= M < 2^31");
  if (D > attamba::kMaxNormDim) return refuse(kUnsupported, name, "D is at most 32768");
  if (!(eps >= 0.f)) return refuse(kInvalid, name, "eps >= 0");
  if ((!y && !res) || (!res_out && !h)) return refuse(kInvalid, name, "y or res, and res_out or h, are required");
  if ((h == nullptr) != (w_pre == nullptr)) return refuse(kInvalid, name, "h and w_pre go together");
  if (!y && (gate || w_post || scale)) return refuse(kInvalid, name, "gate, w_post and scale belong to y");
  if (act != ATTAMBA_ACT_LINEAR && act != ATTAMBA_ACT_SILU && act != ATTAMBA_ACT_SIGMOID)
    return refuse(kInvalid, name, "act is LINEAR, SILU or SIGMOID");
  if (!aligned16(w_post) || !aligned16(scale) || !aligned16(w_pre))
    return refuse(kInvalid, name, "w_post, scale and w_pre are 16-byte aligned");
  const int es = elem_size(dtype), rs = elem_size(res_dtype);
  // an output in place of its input is written by the thread that read it, after the row's last read
  const bool in_place_r = res_out && res_out == res && ldro == ldr, in_place_h = h && h == y && ldh == ldy;
  const Rows rows[] = {{in_place_h ? nullptr : y, M, ldy, D, es, false, "y"},
                       {gate, M, ldg, D, es, false, "gate"},
                       {in_place_r ? nullptr : res, M, ldr, D, rs, false, "res"},
                       {res_out, M, ldro, D, rs, true, "res_out"},
                       {h, M, ldh, D, es, true, "h"}};
  const attamba_status_t st = check_rows(rows, 5, name);
  if (st != ATTAMBA_OK) return st;
  attamba::NormArgs a{};
  a.y = y; a.gate = gate; a.res = res; a.w_post = w_post; a.scale = scale; a.w_pre = w_pre; a.res_out = res_out; a.h = h;
  a.ldy = ldy; a.ldg = ldg; a.ldr = ldr; a.ldro = ldro; a.ldh = ldh;
  a.M = M; a.D = D; a.act = (int32_t)act; a.gate_first = gate_first; a.alpha = alpha; a.eps = eps;
  const cudaError_t e = attamba::launch_block_norm(dtype, res_dtype, a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTAMBA_OK : cuda_fail(e, name);
}

}  // extern "C"
