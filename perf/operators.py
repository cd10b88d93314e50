"""Measured cases of the selective-SSM block operators: their plain forms and the library's calls.

The operators are those a Mamba-style block needs beside the Attamba layer's own scans:

  conv       short causal depthwise convolution over packed prompts, with the carried input window
  conv_step  the same for one token per sequence
  scan       selective state-space scan over packed prompts, with skip, gate and carried state
  scan_step  the same for one token per sequence
  norm       norms after and before a block fused with its gate, residual scale and residual sum

``run`` makes one pass: with ``own`` false in elementary torch operations in 32 bits, with ``own``
true through ``ssm_compressed_chunked_b200.attamba``.  Both update the carried states in place, as a
serving program does, and return the whole outputs and the whole state.  ``exact`` gives the same
values in 64 bits, the recurrences token by token.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTH = {"bf16": 2, "f32": 4}


def listed():
    return [
        # conv: a short prompt's first pass (latency counts), and a packed prefill batch whose input is the
        # left half of the [T, 2 D] input projection
        dict(name="conv_short_prompt", op="conv", dtype="bf16", T=61, D=1024, K=4, S=1, pad=0, halves=1),
        dict(name="conv_packed_prefill", op="conv", dtype="bf16", T=32768, D=2048, K=4, S=11, pad=37, halves=2),
        # conv_step: one request, and a decode batch padded to its graph's size
        dict(name="conv_step_single", op="conv_step", dtype="bf16", B=1, D=2048, K=4, pad=0, slots=4),
        dict(name="conv_step_batch", op="conv_step", dtype="bf16", B=256, D=2048, K=4, pad=5, slots=300),
        # scan: a short prompt, continued chunks of three prompts in fp32, a packed prefill batch of the
        # inference-mask workload's token count and width, and one long prompt with the larger state
        dict(name="scan_short_prompt", op="scan", dtype="bf16", T=61, D=1024, N=16, S=1, pad=0, gate=True),
        dict(name="scan_chunks_f32", op="scan", dtype="f32", T=1029, D=512, N=16, S=3, pad=5, gate=False),
        dict(name="scan_packed_prefill", op="scan", dtype="bf16", T=16384, D=1024, N=16, S=9, pad=21, gate=True),
        dict(name="scan_long_prompt_n32", op="scan", dtype="bf16", T=16384, D=1024, N=32, S=1, pad=0, gate=True),
        # scan_step: one request, and the decode workload's batch and width with padded rows
        dict(name="scan_step_single", op="scan_step", dtype="bf16", B=1, D=1024, N=16, pad=0, slots=4, gate=True),
        dict(name="scan_step_batch", op="scan_step", dtype="bf16", B=256, D=2048, N=16, pad=5, slots=300, gate=True),
        # norm: a decode batch between two blocks, and a prefill with the residual stream in fp32
        dict(name="norm_decode", op="norm", dtype="bf16", res="bf16", M=32, D=2048, gate="none", first=False,
             post=True, pre=True),
        dict(name="norm_prefill", op="norm", dtype="bf16", res="f32", M=16384, D=2048, gate="silu", first=False,
             post=True, pre=True),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("conv", "conv_step", "scan", "scan_step", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "conv":
        D = 8 * _between(rng, 8, 512)
        T = _between(rng, 1, min(65536, (32768 * 2048) // D // (WIDTH[dtype] // 2)))
        S = _between(rng, 1, 40)
        return dict(op=op, dtype=dtype, T=T, D=D, K=rng.choice((2, 3, 4, 4)), S=S, pad=rng.choice((0, 0, rng.randint(1, 64))),
                    halves=rng.choice((1, 2)))
    if op == "conv_step":
        B = _between(rng, 1, 512)
        return dict(op=op, dtype=dtype, B=B, D=8 * _between(rng, 8, 512), K=rng.choice((2, 3, 4, 4)),
                    pad=rng.randint(0, B // 4), slots=B + rng.randint(0, 40))
    if op == "scan":
        N = rng.choice((16, 16, 32))
        D = 8 * _between(rng, 8, 256)
        T = _between(rng, 1, min(32768, (16384 * 1024 * 32) // (D * N)))
        return dict(op=op, dtype=dtype, T=T, D=D, N=N, S=_between(rng, 1, 40), pad=rng.choice((0, 0, rng.randint(1, 64))),
                    gate=rng.random() < 0.7)
    if op == "scan_step":
        N = rng.choice((16, 16, 32))
        B = _between(rng, 1, 512 // (N // 16))
        return dict(op=op, dtype=dtype, B=B, D=8 * _between(rng, 8, 512), N=N, pad=rng.randint(0, B // 4),
                    slots=B + rng.randint(0, 40), gate=rng.random() < 0.7)
    D = 8 * _between(rng, 8, 1024)
    post, pre = rng.choice(((True, True), (True, True), (True, False), (False, True)))
    return dict(op=op, dtype=dtype, res=rng.choice(("bf16", "f32")), M=_between(rng, 1, (16384 * 2048) // (D * WIDTH[dtype] // 2)), D=D,
                gate=rng.choice(("none", "silu", "sigmoid", "linear")), first=rng.random() < 0.4, post=post, pre=pre)


# ---------------------------------------------------------------- inputs
def _sequences(S, total, gen):
    """Offsets [S + 1] of S ragged sequences over `total` tokens; with four or more of them one is empty."""
    w = -np.log(np.maximum(gen.random(S), 1e-9)) + 0.05
    if S >= 4:
        w[S // 2] = 0.0
    cut = np.floor(np.cumsum(w) / w.sum() * total + 0.5).astype(np.int64)
    cut[-1] = total
    if S >= 4:
        cut[S // 2] = cut[S // 2 - 1]
    return np.concatenate(([0], cut))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    host = np.random.default_rng(int(seed))
    dt = TYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s = dict(case=case, op=op)
    if op == "norm":
        M, D = case["M"], case["D"]
        s["y"] = normal(M, D, scale=2.0)
        s["gate"] = normal(M, D) if case["gate"] != "none" else None
        s["res"] = normal(M, D, dtype=TYPES[case["res"]], scale=3.0)
        s["w_post"] = 0.5 + uniform(D) if case["post"] else None
        s["w_pre"] = 0.5 + uniform(D) if case["pre"] else None
        s["alpha"], s["eps"] = 0.7071, 1e-5
        s["res_out"] = torch.zeros(M, D, dtype=TYPES[case["res"]], device=dev)
        s["h"] = torch.zeros(M, D, dtype=dt, device=dev) if case["pre"] else None
        return s

    D = case["D"]
    if op in ("conv", "scan"):
        T, S = case["T"], case["S"]
        total = max(0, T - case["pad"])
        cu = _sequences(S, total, host)
        s["cu"] = torch.from_numpy(cu.astype(np.int32)).to(dev)
        s["T"], s["total"], s["longest"] = T, total, int((cu[1:] - cu[:-1]).max())
        rows, n_slots = T, S + 3
        s["slots"] = torch.from_numpy(host.permutation(n_slots)[:S].astype(np.int32)).to(dev)
        s["cont"] = torch.from_numpy((host.random(S) < 0.5).astype(np.int32)).to(dev)
    else:
        rows, n_slots = case["B"], case["slots"]
        sl = host.permutation(n_slots)[:rows].astype(np.int32)
        if case["pad"]:
            sl[rows - case["pad"]:] = -1     # rows that only fill the batch up
        s["slots"] = torch.from_numpy(sl).to(dev)
        s["rows"] = rows - case["pad"]
    s["n_slots"] = n_slots

    if op in ("conv", "conv_step"):
        K = case["K"]
        wide = normal(rows, case.get("halves", 1) * D)
        s["x"] = wide[:, :D]
        s["w"] = normal(D, K, dtype=torch.float32, scale=K ** -0.5)
        s["bias"] = normal(D, dtype=torch.float32, scale=0.1)
        s["state"] = normal(n_slots, K - 1, D)
    else:
        N = case["N"]
        s["x"] = normal(rows, D)
        s["dt"] = normal(rows, D)
        s["B"], s["C"] = normal(rows, N), normal(rows, N)
        s["z"] = normal(rows, D) if case["gate"] else None
        s["A"] = -torch.exp(uniform(D, N) * math.log(16.0))
        # softplus(bias) log-uniform in [1e-3, 1e-1]
        d0 = torch.exp(uniform(D).double() * math.log(100.0) + math.log(1e-3))
        s["bias"] = (d0 + torch.log(-torch.expm1(-d0))).float()
        s["skip"] = normal(D, dtype=torch.float32)
        s["state"] = normal(n_slots, N, D, dtype=torch.float32)
    s["out"] = torch.zeros(rows, D, dtype=dt, device=dev)
    return s


# ---------------------------------------------------------------- plain forms
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _act(name, v):
    return {"silu": _silu, "sigmoid": lambda u: 1.0 / (1.0 + torch.exp(-u)), "linear": lambda u: u}[name](v)


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _owner(s, total):
    """The sequence that each of the first `total` tokens belongs to, and the first token of it."""
    ends = s["cu"][1:].long()
    seq = torch.searchsorted(ends, torch.arange(total, device=ends.device), right=True)
    return seq, s["cu"].long()[seq]


def _plain_conv(s):
    K = s["w"].shape[1]
    x = s["x"].float()
    old = s["state"][s["slots"].long()].float() * s["cont"].float()[:, None, None]     # [S, K - 1, D]
    back = torch.arange(K, device=x.device) - (K - 1)

    def window(at, first, seq, taps):
        """Inputs at positions at + taps of each sequence; those before its first token from the kept window."""
        pos = at[:, None] + taps[None, :]
        kept = (pos - first[:, None] + (K - 1)).clamp(0, K - 2)
        return torch.where((pos >= first[:, None])[..., None], x[pos.clamp(min=0)], old[seq[:, None], kept])

    total = s["total"]
    if total:
        seq, first = _owner(s, total)
        v = window(torch.arange(total, device=x.device), first, seq, back)
        s["out"][:total] = _silu((v * s["w"].t()[None]).sum(1) + s["bias"]).to(s["out"].dtype)
        cu = s["cu"].long()
        ids = torch.arange(len(cu) - 1, device=x.device)
        s["state"][s["slots"].long()] = window(cu[1:] - 1, cu[:-1], ids, back[1:]).to(s["state"].dtype)
    else:
        s["state"][s["slots"].long()] = old.to(s["state"].dtype)
    return s["out"], s["state"]


def _plain_conv_step(s):
    n = s["rows"]
    sl = s["slots"][:n].long()
    v = torch.cat((s["state"][sl].float(), s["x"][:n].float()[:, None]), dim=1)          # [n, K, D]
    s["out"][:n] = _silu((v * s["w"].t()[None]).sum(1) + s["bias"]).to(s["out"].dtype)
    s["state"][sl] = v[:, 1:].to(s["state"].dtype)
    return s["out"], s["state"]


def _plain_scan(s):
    """h_t = a_t h_{t-1} + b_t as a prefix of pairs (a, b) by doubling: log2(longest sequence) steps over whole
    tensors.  The pairs at sequence starts have a = 0, their b holds the carried state's share."""
    total = s["total"]
    sl = s["slots"].long()
    h0 = s["state"][sl] * s["cont"].float()[:, None, None]                                # [S, N, D]
    if total:
        x = s["x"][:total].float()
        delta = _softplus(s["dt"][:total].float() + s["bias"])
        a = torch.exp(delta[:, None, :] * s["A"].t()[None])                               # [T, N, D]
        b = (delta * x)[:, None, :] * s["B"][:total].float()[:, :, None]
        lens = s["cu"].long()[1:] - s["cu"].long()[:-1]
        some = lens > 0
        starts = s["cu"].long()[:-1][some]
        b[starts] += a[starts] * h0[some]
        a[starts] = 0.0
        o = 1
        while o < s["longest"]:
            b[o:] = b[o:] + a[o:] * b[:-o]
            a[o:] = a[o:] * a[:-o]
            o *= 2
        y = (b * s["C"][:total].float()[:, :, None]).sum(1) + s["skip"] * x
        if s["z"] is not None:
            y = y * _silu(s["z"][:total].float())
        s["out"][:total] = y.to(s["out"].dtype)
        ends = (s["cu"].long()[1:] - 1).clamp(min=0)
        h0 = torch.where(some[:, None, None], b[ends], h0)
    s["state"][sl] = h0
    return s["out"], s["state"]


def _plain_scan_step(s):
    n = s["rows"]
    sl = s["slots"][:n].long()
    x = s["x"][:n].float()
    delta = _softplus(s["dt"][:n].float() + s["bias"])
    h = torch.exp(delta[:, None, :] * s["A"].t()[None]) * s["state"][sl]
    h = h + (delta * x)[:, None, :] * s["B"][:n].float()[:, :, None]
    y = (h * s["C"][:n].float()[:, :, None]).sum(1) + s["skip"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"][:n].float())
    s["out"][:n] = y.to(s["out"].dtype)
    s["state"][sl] = h
    return s["out"], s["state"]


def _plain_norm(s):
    c = s["case"]
    v = s["y"].float()
    if c["gate"] != "none" and c["first"]:
        v = v * _act(c["gate"], s["gate"].float())
    if c["post"]:
        v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + s["eps"]) * s["w_post"]
    if c["gate"] != "none" and not c["first"]:
        v = v * _act(c["gate"], s["gate"].float())
    r = s["res"].float() + s["alpha"] * v
    out = [r.to(s["res"].dtype)]
    if c["pre"]:
        out.append((r * torch.rsqrt((r * r).mean(1, keepdim=True) + s["eps"]) * s["w_pre"]).to(s["y"].dtype))
    return out


# ---------------------------------------------------------------- the library's calls
def _own_run(s):
    from ssm_compressed_chunked_b200 import attamba as A
    op = s["op"]
    if op == "norm":
        c = s["case"]
        act = {"none": A.ACT_SILU, "silu": A.ACT_SILU, "sigmoid": A.ACT_SIGMOID, "linear": A.ACT_LINEAR}[c["gate"]]
        A.block_norm(s["y"], s["res"], s["res_out"], s["h"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                     gate_act=act, gate_first=c["first"], alpha=s["alpha"], eps=s["eps"])
        return [s["res_out"], s["h"]] if c["pre"] else [s["res_out"]]
    if op == "conv_step":
        A.conv_step(s["x"], s["w"], s["bias"], s["state"], s["out"], slots=s["slots"])
        return s["out"], s["state"]
    if op == "scan_step":
        A.scan_step(s["x"], s["dt"], s["bias"], s["A"], s["B"], s["C"], s["state"], s["out"], skip=s["skip"], z=s["z"],
                    slots=s["slots"])
        return s["out"], s["state"]
    if "seqs" not in s:      # the sequence table a serving program keeps beside its batch
        s["seqs"] = A.Seqs(s["cu"], s["T"], slots=s["slots"], cont=s["cont"])
    if op == "conv":
        A.causal_conv(s["x"], s["w"], s["bias"], s["seqs"], s["out"], state=s["state"])
        return s["out"], s["state"]
    if "workspace" not in s:
        size = A.selective_scan_workspace_size(s["T"], s["x"].shape[1], s["A"].shape[1])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["x"].device)
    A.selective_scan(s["x"], s["dt"], s["bias"], s["A"], s["B"], s["C"], s["seqs"], s["out"], skip=s["skip"], z=s["z"],
                     state=s["state"], workspace=s["workspace"])
    return s["out"], s["state"]


def run(state):
    if own:
        return _own_run(state)
    return {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_step": _plain_scan_step,
            "norm": _plain_norm}[state["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; padded rows and unused slots not counted."""
    op, e = case["op"], WIDTH[case["dtype"]]
    if op == "norm":
        M, D, r = case["M"], case["D"], WIDTH[case["res"]]
        gate = case["gate"] != "none"
        per = e + 2 * r + (e if gate else 0) + (e if case["pre"] else 0)
        flops = 2 + (6 if gate else 0) + (4 if case["post"] else 0) + (4 if case["pre"] else 0)
        return {"bytes": M * D * per + 4 * D * (case["post"] + case["pre"]), "flops": M * D * flops}
    D = case["D"]
    rows = max(0, case["T"] - case["pad"]) if op in ("conv", "scan") else case["B"] - case["pad"]
    seqs = case["S"] if op in ("conv", "scan") else rows
    # of a prompt's states half are read (the sequences that continue), all are written
    moved = seqs * (1.5 if op in ("conv", "scan") else 2.0)
    if op in ("conv", "conv_step"):
        K = case["K"]
        return {"bytes": rows * D * 2 * e + moved * (K - 1) * D * e + 4 * D * (K + 1), "flops": rows * D * (2 * K + 5)}
    N = case["N"]
    per = (3 + (1 if case["gate"] else 0)) * e
    return {"bytes": rows * (D * per + 2 * N * e) + moved * N * D * 4 + 4 * D * (N + 2),
            "flops": rows * D * (7 * N + 8 + (5 if case["gate"] else 0))}


# ---------------------------------------------------------------- 64 bits
def _padded(v, s):
    """[T, ...] tokens as [S, longest, ...], and which places hold one."""
    cu = s["cu"].cpu().numpy().astype(np.int64)
    n = s["longest"]
    out = torch.zeros(len(cu) - 1, n, *v.shape[1:], dtype=torch.float64, device=v.device)
    for i in range(len(cu) - 1):
        out[i, :cu[i + 1] - cu[i]] = v[cu[i]:cu[i + 1]].double()
    return out


def _packed(v, s):
    cu = s["cu"].cpu().numpy().astype(np.int64)
    out = s["out"].double()
    for i in range(len(cu) - 1):
        out[cu[i]:cu[i + 1]] = v[i, :cu[i + 1] - cu[i]]
    return out


def _exact_silu(v):
    return v * torch.sigmoid(v)


def _exact_conv(s):
    w, K = s["w"].double(), s["w"].shape[1]
    st = s["state"].double()
    if s["op"] == "conv_step":
        x, n = s["x"].double(), s["rows"]
        y = s["out"].double()
        for i, slot in enumerate(s["slots"].tolist()[:n]):
            line = torch.cat((st[slot], x[i:i + 1]))
            y[i] = _exact_silu((line * w.t()).sum(0) + s["bias"].double())
            st[slot] = line[1:]
        return y, st
    cu, y = s["cu"].tolist(), s["out"].double()
    for i, (slot, cont) in enumerate(zip(s["slots"].tolist(), s["cont"].tolist())):
        x = s["x"][cu[i]:cu[i + 1]].double()
        line = torch.cat((st[slot] * cont, x))
        acc = s["bias"].double().expand(x.shape[0], -1).clone()
        for k in range(K):
            acc += line[k:k + x.shape[0]] * w[:, k]
        y[cu[i]:cu[i + 1]] = _exact_silu(acc)
        st[slot] = line[line.shape[0] - (K - 1):]
    return y, st


def _exact_scan(s):
    A, bias, skip = s["A"].double().t(), s["bias"].double(), s["skip"].double()
    st = s["state"].double()

    def token(h, x, dt, B, C, z):
        delta = torch.logaddexp(dt + bias, torch.zeros_like(dt))
        h = torch.exp(delta[:, None] * A) * h + (delta * x)[:, None] * B[:, :, None]
        y = torch.einsum("bnd,bn->bd", h, C) + skip * x
        return h, y if z is None else y * _exact_silu(z)

    if s["op"] == "scan_step":
        n = s["rows"]
        sl = s["slots"][:n].long()
        y = s["out"].double()
        st[sl], y[:n] = token(st[sl], *(s[k][:n].double() for k in ("x", "dt", "B", "C")),
                              None if s["z"] is None else s["z"][:n].double())
        return y, st
    sl = s["slots"].long()
    h = st[sl] * s["cont"].double()[:, None, None]
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    cols = {k: _padded(s[k], s) for k in ("x", "dt", "B", "C")}
    z = None if s["z"] is None else _padded(s["z"], s)
    y = torch.zeros_like(cols["x"])
    for t in range(s["longest"]):
        nh, y[:, t] = token(h, *(cols[k][:, t] for k in ("x", "dt", "B", "C")), None if z is None else z[:, t])
        h = torch.where((t < lens)[:, None, None], nh, h)
    st[sl] = h
    return _packed(y, s), st


def _exact_norm(s):
    c = s["case"]
    v = s["y"].double()
    gate = {"none": lambda u: None, "silu": _exact_silu, "sigmoid": torch.sigmoid, "linear": lambda u: u}[c["gate"]](
        None if s["gate"] is None else s["gate"].double())
    if gate is not None and c["first"]:
        v = v * gate
    if c["post"]:
        v = v / (v.square().sum(1, keepdim=True) / v.shape[1] + s["eps"]).sqrt() * s["w_post"].double()
    if gate is not None and not c["first"]:
        v = v * gate
    r = s["res"].double() + s["alpha"] * v
    out = [r]
    if c["pre"]:
        out.append(r / (r.square().sum(1, keepdim=True) / r.shape[1] + s["eps"]).sqrt() * s["w_pre"].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "conv_step": _exact_conv, "scan": _exact_scan, "scan_step": _exact_scan,
            "norm": _exact_norm}[s["op"]](s)
