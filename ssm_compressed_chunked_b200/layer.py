"""The prefill hot path as three C-ABI calls on preallocated device buffers,
and the whole layer with its projections around it.

    chunk_index  ->  kv_ssm_scan (K and V, plus the chunk-end rows Kc, Vc)  ->  chunk_attn_fwd

    Layer:  x  --proj_gemm-->  q, dt_K, dt_V, B_K, C_K, B_V, C_V  --hot path-->  O  --proj_gemm-->  y = O W_O

Beside it, the same selective SSM uncompressed, as a Mamba block's mixer, and the residual block around either:

    SsmMixer:  h  --proj_gemm-->  x, z;  x  --causal_conv-->  u  --proj_gemm-->  dt, B, C;
               selective_scan(u, dt, A, B, C, skip, z)  --proj_gemm-->  y
    Block:     r  --block_norm-->  h  --mixer-->  y  --block_norm-->  r + alpha scale norm(y), and the next block's h

Only buffer allocation happens here (torch, once); every step of the path runs
in libattamba.so.
"""

import torch

from . import attamba as A


class Prefill:
    """Device buffers of one prefill and the three calls over them.

    ``alloc(shape, dtype)`` returns each output buffer (default: uninitialised
    device memory); a caller can hand in its own, e.g. pre-filled memory."""

    def __init__(self, B, n, D, H, dh, N, n_chunks, dtype, device="cuda", alloc=None):
        self.B, self.n, self.D, self.H, self.dh, self.N = B, n, D, H, dh, N
        self.n_chunks = n_chunks
        self.dtype = dtype
        T = B * n
        if alloc is None:
            alloc = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        self.index = A.Index(n_chunks, B, n, device, alloc=alloc)
        self.K = alloc((T, D), dtype)
        self.V = alloc((T, D), dtype)
        self.Kc = alloc((n_chunks, D), dtype)
        self.Vc = alloc((n_chunks, D), dtype)
        self.O = alloc((T, H, dh), dtype)
        self.lse = alloc((B, H, n), torch.float32)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def index_step(self, cu_in, P, offset, L, mode, stream=None):
        A.chunk_index(cu_in, self.n_chunks, self.B, self.n, P, offset, L, mode, self.index, self.status, stream)

    def scan_step(self, x, dt_k, dt_v, bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, stream=None):
        A.kv_ssm_scan(x, dt_k, dt_v, bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, self.index.cu,
                      self.n_chunks, self.K, self.V, self.Kc, self.Vc, self.status, stream)

    def attn_step(self, q, scale, stream=None):
        H, dh = self.H, self.dh
        A.chunk_attn_fwd(q, self.K.view(-1, H, dh), self.V.view(-1, H, dh), self.Kc.view(-1, H, dh),
                         self.Vc.view(-1, H, dh), self.index, scale, self.O, self.lse, self.status, stream)

    def forward(self, x, q, dt_k, dt_v, bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, cu_in, P, offset, L,
                mode, scale, stream=None):
        self.index_step(cu_in, P, offset, L, mode, stream)
        self.scan_step(x, dt_k, dt_v, bias_k, bias_v, A_k, A_v, B_k, C_k, B_v, C_v, stream)
        self.attn_step(q, scale, stream)
        return self.O


def n_chunks_of(cfg, cu=None):
    """Chunk count of a workload: uniform from the library's count, variable from its cu array."""
    if cfg.varlen is None:
        return cfg.B * A.uniform_chunk_count(cfg.n, cfg.P, cfg.offset)
    return len(cu) - 1


def mode_code(mode):
    return A.MASK_TRAIN if mode == "train" else A.MASK_TEST


# the layer's input projections, in the column order of the one GEMM that computes them
INPUT_PROJECTIONS = ("W_Q", "W_dtK", "W_dtV", "W_BK", "W_CK", "W_BV", "W_CV")


class Layer:
    """One Attamba layer forward, y = Attn(q, K, V) W_O, on preallocated device buffers.

    pith.science review of Attamba, "Core claim": the keys and values come from
    two SSMs over the layer input (K = SSM_K(x), V = SSM_V(x)) in place of W_K
    and W_V, while the query and output projections stay; "Assumptions & free
    parameters": each SSM is Mamba's selective SSM, whose step and B, C are
    projections of its input.  So x is projected seven ways (q, dt_K, dt_V, B_K,
    C_K, B_V, C_V) by one GEMM whose column segments land in the arrays the hot
    path reads, the hot path gives O, and a second GEMM gives y = O W_O.

    ``weights`` maps each name of INPUT_PROJECTIONS and "W_O" to a bf16 matrix in
    [out, in] layout (W_Q [H dh, D]; W_dtK, W_dtV [D, D]; W_BK ... W_CV [N, D];
    W_O [D, H dh]) and "bias_k", "bias_v" [D], "A_k", "A_v" [D, N] to fp32; all on
    the layer's device.  The chunking is uniform (P, offset) unless ``forward``
    gets chunk offsets ``cu_in`` (then ``n_chunks`` must be their count);
    ``mode`` is MASK_TEST or MASK_TRAIN.

    Decoding (pith.science review, "Core claim": the inference cache holds the
    chunk boundary states, and "If this is right": P = 8 with 64 leading tokens)
    continues a uniform-chunk prefill one token at a time under M_test:
    ``new_cache`` or ``cache_from_prefill`` gives the cache, ``decode_step`` maps
    x_t to y_t."""

    def __init__(self, B, n, D, H, dh, N, weights, P, offset, L, mode, scale, n_chunks=None, device="cuda",
                 alloc=None):
        bf = torch.bfloat16
        self.B, self.n, self.D, self.H, self.dh, self.N = B, n, D, H, dh, N
        self.P, self.offset, self.L, self.mode, self.scale = P, offset, L, mode, scale
        T = B * n
        shapes = {"W_Q": (H * dh, D), "W_dtK": (D, D), "W_dtV": (D, D), "W_BK": (N, D), "W_CK": (N, D),
                  "W_BV": (N, D), "W_CV": (N, D), "W_O": (D, H * dh)}
        for name, shape in shapes.items():
            w = weights[name]
            if tuple(w.shape) != shape or w.dtype != bf:
                raise A.AttambaError(f"{name} must be bf16 {shape}, got {w.dtype} {tuple(w.shape)}")
        self.W_in = torch.cat([weights[k] for k in INPUT_PROJECTIONS], dim=0).contiguous()
        self.W_O = weights["W_O"].contiguous()
        self.bias_k, self.bias_v = weights["bias_k"], weights["bias_v"]
        self.A_k, self.A_v = weights["A_k"], weights["A_v"]
        if alloc is None:
            alloc = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        widths = [shapes[k][0] for k in INPUT_PROJECTIONS]
        self.proj, c = [], 0
        for w in widths:
            self.proj.append((alloc((T, w), bf), c))
            c += w
        if n_chunks is None:
            n_chunks = B * A.uniform_chunk_count(n, P, offset)
        self.prefill = Prefill(B, n, D, H, dh, N, n_chunks, bf, device=device, alloc=alloc)
        self.y = alloc((T, D), bf)
        self.status = self.prefill.status
        self.device = self.status.device
        self._step = None   # decode buffers, made by the first decode_step

    @property
    def projections(self):
        """The projected activations, by the names of INPUT_PROJECTIONS without the "W_"."""
        return {k[2:]: t for k, (t, _) in zip(INPUT_PROJECTIONS, self.proj)}

    # ---------------------------------------------------------------- decode (M_test, uniform chunks)
    def new_cache(self, cap, device=None):
        """An empty decode cache (every sequence at position 0) with room for ``cap`` chunk-end rows
        per sequence and the layer's L most recent tokens, chunked like the layer (P, offset); on the
        layer's device unless ``device`` says otherwise."""
        if self.L < 1:
            raise A.AttambaError("decoding keeps the L >= 1 most recent tokens; this layer has L = 0")
        device = self.W_in.device if device is None else device
        B, H, dh, N, D, L = self.B, self.H, self.dh, self.N, self.D, self.L
        bf, i32 = torch.bfloat16, torch.int32
        z = lambda *shape, dt=bf: torch.zeros(*shape, dtype=dt, device=device)  # noqa: E731
        return A.Cache(z(2, B, N, D, dt=torch.float32), z(B, H, cap, dh), z(B, H, cap, dh), z(B, cap, dt=i32),
                       z(B, H, L, dh), z(B, H, L, dh), z(B, dt=i32), z(B, dt=i32), self.P, self.offset)

    def cache_from_prefill(self, cache, x, stream=None):
        """Fill ``cache`` with what the last ``forward`` (over x, all n tokens of each sequence, uniform
        chunks) leaves for decoding position n onwards: its chunk-end keys and values, its last L
        tokens and the SSM states after token n - 1."""
        B, n, H, dh = self.B, self.n, self.H, self.dh
        pf = self.prefill
        _, dt_k, dt_v, B_k, C_k, B_v, C_v = (t for t, _ in self.proj)
        A.cache_from_prefill(cache, pf.K.view(B, n, H, dh), pf.V.view(B, n, H, dh), x, dt_k, dt_v, self.bias_k,
                             self.bias_v, self.A_k, self.A_v, B_k, C_k, B_v, C_v, n, self.status, stream)

    def decode_step(self, cache, x_t, stream=None):
        """One new token per sequence under the inference mask M_test: x_t [B, D] bf16 -> y_t [B, D]
        (the layer's own buffer).  The same seven projections as ``forward`` (one GEMM of B rows), the
        decode step over ``cache`` (which it advances by one position), then W_O."""
        B, H, dh, D = self.B, self.H, self.dh, self.D
        bf = torch.bfloat16
        if self._step is None:
            dev = self.W_in.device
            self._step, c = [], 0
            for (t, _) in self.proj:
                self._step.append((torch.empty(B, t.shape[1], dtype=bf, device=dev), c))
                c += t.shape[1]
            self.o_t = torch.empty(B, H, dh, dtype=bf, device=dev)
            self.y_t = torch.empty(B, D, dtype=bf, device=dev)
            self._ws = {}
        size = A.decode_workspace_size(cache)
        if size not in self._ws:
            self._ws[size] = torch.empty(size, dtype=torch.uint8, device=self.W_in.device)
        q, dt_k, dt_v, B_k, C_k, B_v, C_v = (t for t, _ in self._step)
        A.proj_gemm(x_t, self.W_in, self._step, self.status, stream)
        A.decode_step(cache, q.view(B, H, dh), x_t, dt_k, dt_v, self.bias_k, self.bias_v, self.A_k, self.A_v, B_k,
                      C_k, B_v, C_v, self.scale, self.o_t, self._ws[size], self.status, stream)
        A.proj_gemm(self.o_t.view(B, H * dh), self.W_O, [(self.y_t, 0)], self.status, stream)
        return self.y_t

    @property
    def step_projections(self):
        """The last decode step's projections, named like ``projections``."""
        if self._step is None:
            raise A.AttambaError("no decode step has run on this layer")
        return {k[2:]: t for k, (t, _) in zip(INPUT_PROJECTIONS, self._step)}

    def forward(self, x, cu_in=None, stream=None):
        """x [B n, D] bf16 -> y [B n, D] bf16 (the layer's own buffer)."""
        T, H, dh = self.B * self.n, self.H, self.dh
        q, dt_k, dt_v, B_k, C_k, B_v, C_v = (t for t, _ in self.proj)
        A.proj_gemm(x, self.W_in, self.proj, self.status, stream)
        pf = self.prefill
        pf.index_step(cu_in, self.P if cu_in is None else 1, self.offset, self.L, self.mode, stream)
        pf.scan_step(x, dt_k, dt_v, self.bias_k, self.bias_v, self.A_k, self.A_v, B_k, C_k, B_v, C_v, stream)
        pf.attn_step(q.view(T, H, dh), self.scale, stream)
        A.proj_gemm(pf.O.view(T, H * dh), self.W_O, [(self.y, 0)], self.status, stream)
        return self.y


def _check_device(own, t, stream, what):
    """The projections launch on the current device and the SSM block's operators on their tensors': tensors, stream and
    current device must be where ``own`` is."""
    if t.device != own:
        raise A.AttambaError(f"{what} is on {own}, its input on {t.device}")
    if own.type == "cuda":
        if torch.cuda.current_device() != own.index:
            raise A.AttambaError(f"{what}: {own} is not the current device")
        if stream is not None and stream.device_index != own.index:
            raise A.AttambaError(f"{what} is on {own}, the stream is on cuda:{stream.device_index}")


class SsmMixer:
    """A Mamba block's mixer: the layer's selective SSM over whole sequences, with its short convolution, skip
    and gate.

    pith.science review of Attamba, "Assumptions & free parameters": the SSM is Mamba's selective SSM (Section
    3.2, Eq. 3).  Here it is not chunked: its state runs through each sequence and is carried from call to call.
    One GEMM gives the SSM input and its gate, the convolution (with SiLU) the scan's input u, a second GEMM the
    step and B, C from u, the scan its gated output, a third GEMM y.  The step's projection is full-rank, as the
    layer's are: a checkpoint whose step goes through a low rank r (dt = W_dt W_r u) has the two multiplied out into
    the first Di rows of W_x, and pays Di x Di a token for them instead of 2 r Di.

    ``weights``: W_in [2 Di, D], W_x [Di + 2 N, Di] (rows dt, B, C), W_O [D, Di] bf16 in [out, in] layout; conv_w
    [Di, K], A [Di, N] f32; conv_b, bias (of the step), skip [Di] f32 or absent.  D and Di are multiples of 64.
    ``max_tokens`` bounds a call's token rows; the buffers are made once.  Rows of no sequence (behind the last
    prompt, or with slot -1 in a step) come back as zeros.  Calls are made with the mixer's device current."""

    def __init__(self, D, Di, N, K, weights, max_tokens, device="cuda", alloc=None):
        bf, f32 = torch.bfloat16, torch.float32
        shapes = {"W_in": ((2 * Di, D), bf), "W_x": ((Di + 2 * N, Di), bf), "W_O": ((D, Di), bf), "conv_w": ((Di, K), f32),
                  "A": ((Di, N), f32), "conv_b": ((Di,), f32), "bias": ((Di,), f32), "skip": ((Di,), f32)}
        for name, (shape, dt) in shapes.items():
            w = weights.get(name)
            if w is None and name in ("conv_b", "bias", "skip"):
                continue
            if w is None or tuple(w.shape) != shape or w.dtype != dt:
                got = "none" if w is None else f"{w.dtype} {tuple(w.shape)}"
                raise A.AttambaError(f"{name} must be {dt} {shape}, got {got}")
        self.w = {k: (weights[k].contiguous() if weights.get(k) is not None else None) for k in shapes}
        self.D, self.Di, self.N, self.K, self.max_tokens = D, Di, N, K, max_tokens
        if alloc is None:
            alloc = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        widths = dict(x=Di, z=Di, u=Di, dt=Di, B=N, C=N, s=Di, y=D)
        self.buf = {k: alloc((max_tokens, n), bf) for k, n in widths.items()}
        self.workspace = torch.empty(A.selective_scan_workspace_size(max_tokens, Di, N), dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = self.status.device
        for name, t in self.w.items():
            if t is not None and t.device != self.device:
                raise A.AttambaError(f"{name} must be on {self.device}, got {t.device}")
        if any(b.device != self.device for b in self.buf.values()):
            raise A.AttambaError(f"alloc must give buffers on {self.device}")

    def new_state(self, slots):
        """Carried states of ``slots`` sequences, all at zero: (convolution window, SSM state)."""
        dev = self.w["A"].device
        return (torch.zeros(slots, self.K - 1, self.Di, dtype=torch.bfloat16, device=dev),
                torch.zeros(slots, self.N, self.Di, dtype=torch.float32, device=dev))

    def _rows(self, T):
        if not 1 <= T <= self.max_tokens:
            raise A.AttambaError(f"{T} token rows; this mixer holds 1 to {self.max_tokens}")
        return {k: b[:T] for k, b in self.buf.items()}

    def _ends(self, h, b, stream):
        """The input GEMM and a function for the two behind the convolution and behind the scan."""
        A.proj_gemm(h, self.w["W_in"], [(b["x"], 0), (b["z"], self.Di)], self.status, stream)
        Di, N = self.Di, self.N
        return (lambda: A.proj_gemm(b["u"], self.w["W_x"], [(b["dt"], 0), (b["B"], Di), (b["C"], Di + N)], self.status, stream),
                lambda: A.proj_gemm(b["s"], self.w["W_O"], [(b["y"], 0)], self.status, stream))

    def forward(self, h, seqs, state=None, stream=None):
        """h [T, D] bf16 over the sequences of ``seqs`` (attamba.Seqs) -> y [T, D] (the mixer's own buffer); ``state``
        as from new_state, updated in place."""
        _check_device(self.device, h, stream, "this mixer")
        b, w = self._rows(h.shape[0]), self.w
        win, ssm = (None, None) if state is None else state
        steps, out = self._ends(h, b, stream)
        A.causal_conv(b["x"], w["conv_w"], w["conv_b"], seqs, b["u"], state=win, status=self.status, stream=stream)
        steps()
        A.selective_scan(b["u"], b["dt"], w["bias"], w["A"], b["B"], b["C"], seqs, b["s"], skip=w["skip"], z=b["z"],
                         state=ssm, workspace=self.workspace, status=self.status, stream=stream)
        A.clear_rows(b["s"], seqs=seqs, stream=stream)      # W_O makes zeros of zeros
        out()
        return b["y"]

    def decode_step(self, state, h_t, slots=None, stream=None):
        """One new token per sequence: h_t [B, D] bf16 -> y_t [B, D]; ``slots`` [B] int32 names the state rows."""
        _check_device(self.device, h_t, stream, "this mixer")
        b, w = self._rows(h_t.shape[0]), self.w
        win, ssm = state
        steps, out = self._ends(h_t, b, stream)
        A.conv_step(b["x"], w["conv_w"], w["conv_b"], win, b["u"], slots=slots, status=self.status, stream=stream)
        steps()
        A.scan_step(b["u"], b["dt"], w["bias"], w["A"], b["B"], b["C"], ssm, b["s"], skip=w["skip"], z=b["z"], slots=slots,
                    status=self.status, stream=stream)
        if slots is not None:
            A.clear_rows(b["s"], slots=slots, stream=stream)
        out()
        return b["y"]


class Block:
    """A residual block around a mixer (``Layer`` or ``SsmMixer``): r + alpha scale norm(mixer(norm(r))).

    ``w_pre`` [D] f32 is the norm ahead of the mixer, ``w_post`` (or None) the norm behind it, ``scale`` (or None)
    a per-channel residual scale beside the number ``alpha``.  The residual stream r (bf16 or f32) is updated in
    place.  The pass that adds y to r also makes the next block's input: hand its ``w_pre`` over as ``next_norm``
    and give the returned h to the next block, whose own first norm then falls away.  Where the mixer gives zeros
    (``SsmMixer``: rows of no sequence) r stays as it was (with eps > 0, whose norm of zeros is zero).

    ``h`` is what the mixer read in the block's last ``forward`` (handed in or made here): around a Layer it is the
    x of ``Layer.cache_from_prefill``.  A block that makes its input itself keeps the buffers of it, one for
    ``forward`` and one for ``decode_step``: like the mixer's own, they serve one call after the other, so calls
    of a block on several streams are ordered by events."""

    def __init__(self, mixer, w_pre, w_post=None, scale=None, alpha=1.0, eps=1e-5):
        self.mixer, self.w_pre, self.w_post, self.scale, self.alpha, self.eps = mixer, w_pre, w_post, scale, alpha, eps
        self.h = None
        self._prompt, self._step = [], []   # input buffers, the last one of a width the largest

    def _buffer(self, kept, r, first, stream):
        """r.shape rows of bf16 that stay the block's.  Made on the stream that uses them, so that no other stream's
        pending work holds the memory; freed with the block alone, as a captured graph may hold an address."""
        n, D = r.shape
        fit = [b for b in kept if b.shape[1] == D and b.device == r.device]   # others are left from refused calls
        if not fit or fit[-1].shape[0] < n:
            n = max(n, first if not fit else min(2 * fit[-1].shape[0], getattr(self.mixer, "max_tokens", n)))
            with torch.cuda.stream(stream):
                kept.append(torch.empty(n, D, dtype=torch.bfloat16, device=r.device))
            fit = kept
        return fit[-1][:r.shape[0]]

    def _input(self, r, h, kept, first, stream):
        if len(r.shape) != 2:
            raise A.AttambaError(f"r must be [rows, D], got {list(r.shape)}")
        _check_device(getattr(self.mixer, "device", r.device), r, stream, "this block")
        if h is None:
            h = self._buffer(kept, r, first, stream)
            A.block_norm(None, r, h=h, w_pre=self.w_pre, eps=self.eps, stream=stream)
        return h

    def _join(self, y, r, next_norm, stream):
        h = None if next_norm is None else y      # the next input takes y's place
        A.block_norm(y, r, res_out=r, h=h, w_post=self.w_post, w_pre=next_norm, scale=self.scale, alpha=self.alpha,
                     eps=self.eps, stream=stream)
        return r, h

    def forward(self, r, *args, h=None, next_norm=None, stream=None, **kw):
        """r [T, D] -> (r updated, the next block's h or None); the other arguments are the mixer's ``forward``'s."""
        self.h = self._input(r, h, self._prompt, getattr(self.mixer, "max_tokens", 0), stream)
        y = self.mixer.forward(self.h, *args, stream=stream, **kw)
        return self._join(y, r, next_norm, stream)

    def decode_step(self, cache, r, *args, h=None, next_norm=None, stream=None, **kw):
        """The same for one new token per sequence, through the mixer's ``decode_step``."""
        y = self.mixer.decode_step(cache, self._input(r, h, self._step, 0, stream), *args, stream=stream, **kw)
        return self._join(y, r, next_norm, stream)
