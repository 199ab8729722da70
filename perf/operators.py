"""Cases of the operators a linear-recurrence layer needs around its state scan.

Three operators, each forward, with its gradients, and in its serving form:

* ``conv``: the short causal depthwise convolution over the projected channels;
* ``scan``: the selective state space scan (scalar decay per head);
* ``norm``: the root-mean-square norm with the residual's addition, also with
  its output in 8 bits.

``run`` computes a case either from elementary torch operations (``own``
false) or with this package's kernels (``own`` true); ``exact`` computes it
from the definitions in 64 bits.
"""
import math

import numpy as np
import torch
import torch.nn.functional as F

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
FP8_MAX = 448.0
INT8_MAX = 127.0
TINY = 2.0 ** -126        # smallest scale of a quantised row
CHUNK = 64                # tokens per chunk of the plain chunked scan


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one decode step of 256 sequences: the q, k and v channels of 32 heads of 128
        dict(name="conv_step_B256", op="conv", mode="step", dtype="bf16", B=256, T=1, D=12288, W=4,
             bias=False, silu=True, state=True, lens=""),
        # a ragged batch of prompts packed into one row, channels that no vector divides,
        # continued from cached states
        dict(name="conv_prompts_odd", op="conv", mode="fwd", dtype="fp16", B=1, T=18062, D=2505, W=4,
             bias=True, silu=True, state=True, lens="4001,1,350,2903,0,3700,2618,4489"),
        # the convolution of a training step at the benchmark's tokens and heads
        dict(name="conv_train", op="conv", mode="train", dtype="bf16", B=2, T=4096, D=12288, W=4,
             bias=True, silu=True, state=False, lens=""),
        # the norm before a projection in 8 bits, a few decode rows (latency)
        dict(name="norm_fp8_step", op="norm", mode="quant", dtype="bf16", rows=8, D=4096,
             residual="same", quant="fp8", group=0),
        # the same for a prompt, scales per 128 columns
        dict(name="norm_fp8_prompt", op="norm", mode="quant", dtype="bf16", rows=16384, D=4096,
             residual="same", quant="fp8", group=128),
        # an odd width, residual stream in 32 bits
        dict(name="norm_odd", op="norm", mode="fwd", dtype="fp16", rows=4099, D=5003,
             residual="fp32", quant="", group=0),
        # a training step's norm with the residual in the activations' type
        dict(name="norm_train", op="norm", mode="train", dtype="bf16", rows=8192, D=4096,
             residual="same", quant="", group=0),
        # one decode step of one sequence (latency)
        dict(name="scan_step_B1", op="scan", mode="step", dtype="bf16", B=1, T=1, H=32, G=1, P=64,
             N=128, state=True, skip=True, lens=""),
        # one decode step at serving size
        dict(name="scan_step_B256", op="scan", mode="step", dtype="bf16", B=256, T=1, H=32, G=16,
             P=128, N=128, state=True, skip=True, lens=""),
        # packed prompts of unequal lengths, continued from cached states
        dict(name="scan_prompts", op="scan", mode="fwd", dtype="fp16", B=1, T=18062, H=32, G=1, P=64,
             N=128, state=True, skip=True, lens="4001,1,350,2903,0,3700,2618,4489"),
        # one long prompt: few sequences, parallel only along its tokens
        dict(name="scan_long", op="scan", mode="fwd", dtype="bf16", B=1, T=65536, H=32, G=8, P=64,
             N=128, state=False, skip=True, lens=""),
        # a training step at the benchmark's tokens and heads, grouped B and C
        dict(name="scan_train", op="scan", mode="train", dtype="bf16", B=2, T=4096, H=32, G=16,
             P=128, N=128, state=True, skip=True, lens=""),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(rng, T):
    """Packed lengths that sum to T, empty and one-token sequences among them."""
    k = rng.randint(1, min(9, T))
    cuts = sorted(rng.randint(0, T) for _ in range(k - 1))
    edges = [0] + cuts + [T]
    return ",".join(str(b - a) for a, b in zip(edges, edges[1:]))


def draw(rng):
    kind = rng.choice(["conv_step", "conv_fwd", "conv_train", "norm_quant", "norm_fwd",
                       "norm_train", "scan_step", "scan_fwd", "scan_train"])
    op, mode = kind.split("_")
    if op == "norm":
        D = _log_int(rng, 64, 16384)
        rows = _log_int(rng, 1, max(1, (1 << 25) // D))
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        quant = rng.choice(["fp8", "fp8", "int8"]) if mode == "quant" else ""
        return dict(op=op, mode=mode, dtype=dtype, rows=rows, D=D,
                    residual=rng.choice(["none", "same", "fp32"]), quant=quant,
                    group=rng.choice([0, 128]) if quant else 0)
    if op == "conv":
        D = _log_int(rng, 64, 12288)
        W = rng.choice([2, 3, 4, 4, 4])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        bias, silu = rng.random() < 0.5, rng.random() < 0.8
        if mode == "step":
            return dict(op=op, mode=mode, dtype=dtype, B=_log_int(rng, 1, 256), T=rng.choice([1, 1, 1, 3]),
                        D=D, W=W, bias=bias, silu=silu, state=True, lens="")
        T = _log_int(rng, 1, max(64, (1 << 24) // D))
        packed = rng.random() < 0.5
        B = 1 if packed else rng.randint(1, 4)
        return dict(op=op, mode=mode, dtype=dtype, B=B, T=T, D=D, W=W, bias=bias, silu=silu,
                    state=rng.random() < 0.5, lens=_lens(rng, T) if packed else "")
    P, N = rng.choice([64, 128]), rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 8])
    H = G * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "fp16"])
    skip = rng.random() < 0.7
    if mode == "step":
        return dict(op=op, mode=mode, dtype=dtype, B=_log_int(rng, 1, 256), T=rng.choice([1, 1, 1, 4]),
                    H=min(H, 32), G=G, P=P, N=N, state=True, skip=skip, lens="")
    T = _log_int(rng, 1, 8192 * 20 // H if mode == "fwd" else 4096 * 20 // H)
    packed = rng.random() < 0.5
    B = 1 if packed else rng.randint(1, 2)
    return dict(op=op, mode=mode, dtype=dtype, B=B, T=T, H=H, G=G, P=P, N=N,
                state=rng.random() < 0.5, skip=skip, lens=_lens(rng, T) if packed else "")


# ---- inputs -------------------------------------------------------------------

def _lens_of(case):
    return [int(v) for v in case["lens"].split(",")] if case["lens"] else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0, mean=0.0, to=dtype):
        x = torch.randn(*shape, device="cuda", generator=gen)
        return x.mul_(std).add_(mean).to(to)

    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    s = {"case": dict(case)}
    train = case["mode"] == "train"
    if case["op"] == "norm":
        rows, D = case["rows"], case["D"]
        rdt = {"none": None, "same": dtype, "fp32": torch.float32}[case["residual"]]
        s["x"] = randn(rows, D)
        s["residual"] = None if rdt is None else randn(rows, D, std=2.0, to=rdt)
        s["weight"] = randn(D, std=0.2, mean=1.0)
        if train:
            s["dy"] = randn(rows, D)
            s["dres"] = None if rdt is None else randn(rows, D, to=rdt)
            s["leaves"] = [t for t in (s["x"], s["residual"], s["weight"]) if t is not None]
        for t in s.get("leaves", ()):
            t.requires_grad_(True)
        return s

    lens = _lens_of(case)
    s["cu_cpu"] = None
    n_seq = case["B"]
    if lens is not None:
        s["cu_cpu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
        n_seq = len(lens)
    s["cu"] = None if lens is None else s["cu_cpu"].cuda()
    B, T = case["B"], case["T"]
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        s["x"] = randn(B, T, D)
        s["weight"] = randn(D, W, std=W ** -0.5)
        s["bias"] = randn(D, std=0.1) if case["bias"] else None
        s["state"] = randn(n_seq, W - 1, D) if case["state"] else None
        s["activation"] = "silu" if case["silu"] else None
        if train:
            s["dy"] = randn(B, T, D)
            s["dstate"] = randn(n_seq, W - 1, D) if case["state"] else None
            s["leaves"] = [t for t in (s["x"], s["weight"], s["bias"], s["state"]) if t is not None]
    else:
        H, G, P, N = case["H"], case["G"], case["P"], case["N"]
        # x, B and C are slices of one convolution's output, as a layer has them
        width = H * P + 2 * G * N
        xbc = F.silu(randn(B, T, width, to=torch.float32)).to(dtype)
        xs, bs, cs = torch.split(xbc, [H * P, G * N, G * N], dim=-1)
        s["x"] = xs.unflatten(-1, (H, P))
        s["B"] = bs.unflatten(-1, (G, N))
        s["C"] = cs.unflatten(-1, (G, N))
        s["dt"] = randn(B, T, H)
        # parameters of a Mamba-2 style initialisation: decay rates 1..16, step
        # sizes about 0.001..0.1; a bf16 / fp16 model in training holds them in its type
        pt = dtype if train else torch.float32
        s["A_log"] = torch.log(rand(H) * 15 + 1).to(pt)
        dt0 = torch.exp(rand(H) * math.log(100.0) + math.log(0.001))
        s["dt_bias"] = torch.log(torch.expm1(dt0)).to(pt)
        s["D"] = randn(H, std=0.2, mean=1.0, to=pt) if case["skip"] else None
        s["state"] = randn(n_seq, H, N, P, std=0.1, to=torch.float32) if case["state"] else None
        if train:
            # gradients of the slices are asked for, so they are leaves of their own
            s["x"], s["B"], s["C"] = (s[k].detach() for k in ("x", "B", "C"))
            s["dy"] = randn(B, T, H, P)
            s["dstate"] = randn(n_seq, H, N, P, std=0.1, to=torch.float32) if case["state"] else None
            s["leaves"] = [s[k] for k in ("x", "dt", "A_log", "B", "C", "D", "dt_bias", "state")
                           if s[k] is not None]
    for t in s.get("leaves", ()):
        t.requires_grad_(True)
    return s


# ---- the plain forms ------------------------------------------------------------

def _padded(x, cu, cu_cpu):
    """[sequences, longest, ...] from packed [1, T, ...] (zeros behind each
    sequence's end); a dense batch as it is."""
    if cu is None:
        return x
    longest = max(1, int((cu_cpu[1:] - cu_cpu[:-1]).max()))
    pos = torch.arange(longest, device=x.device)
    cu = cu.long()
    live = pos[None] < (cu[1:] - cu[:-1])[:, None]
    idx = torch.where(live, cu[:-1, None] + pos[None], 0)
    rows = x[0][idx]
    return rows * live.reshape(live.shape + (1,) * (x.dim() - 2)).to(rows.dtype)


def _packed(y, cu, T):
    """[1, T, ...] back from the padded sequences."""
    if cu is None:
        return y
    cu = cu.long()
    t = torch.arange(T, device=y.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return y[seq, t - cu[seq]][None]


def _plain_conv(x, weight, bias, state, silu, cu, cu_cpu):
    T, D, W = x.shape[1], x.shape[2], weight.shape[1]
    xp = _padded(x, cu, cu_cpu)
    n, L = xp.shape[0], xp.shape[1]
    before = xp.new_zeros(n, W - 1, D) if state is None else state
    ext = torch.cat([before, xp], dim=1)
    z = (ext.unfold(1, W, 1) * weight).sum(-1)
    if bias is not None:
        z = z + bias
    y = _packed(z * torch.sigmoid(z) if silu else z, cu, T)
    if cu is None:
        last = ext[:, L:]
    else:
        at = (cu[1:] - cu[:-1]).long()[:, None] + torch.arange(W - 1, device=x.device)[None]
        last = ext[torch.arange(n, device=x.device)[:, None], at]
    return y, last


def _plain_scan(x, dt, A_log, Bm, Cm, D, dt_bias, state, cu, cu_cpu):
    T = x.shape[1]
    R = x.shape[2] // Bm.shape[2]
    xp, bp, cp = (_padded(v, cu, cu_cpu) for v in (x, Bm, Cm))
    step = F.softplus(dt.double() + dt_bias.double())
    step = _padded(step, cu, cu_cpu)
    n, L = xp.shape[0], xp.shape[1]
    Q = min(CHUNK, L)
    pad = (-L) % Q
    # [n, heads or groups, chunks, chunk, size]
    cut = lambda v: F.pad(v, (0, 0, 0, 0, 0, pad)).unflatten(1, (-1, Q)).permute(0, 3, 1, 2, 4)  # noqa: E731
    xc, bc, cc = cut(xp), cut(bp), cut(cp)
    sc = F.pad(step, (0, 0, 0, pad)).unflatten(1, (-1, Q)).permute(0, 3, 1, 2)
    g = -torch.exp(A_log.double())[None, :, None, None] * sc
    cum = torch.cumsum(g, -1)                                        # within the chunk, 64 bits
    nc = cum.shape[2]
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp(torch.where(low, cum[..., :, None] - cum[..., None, :], -torch.inf)).float()
    sf = sc.float()
    scores = torch.matmul(cc, bc.transpose(-1, -2).contiguous()).repeat_interleave(R, dim=1)
    y = torch.matmul(scores * decay * sf[..., None, :], xc)
    w = (torch.exp(cum[..., -1:] - cum) * sc).float()
    bh, ch = bc.repeat_interleave(R, dim=1), cc.repeat_interleave(R, dim=1)
    local = torch.matmul(bh.transpose(-1, -2).contiguous(), xc * w[..., None])   # [n, H, nc, N, P]
    total = F.pad(torch.cumsum(cum[..., -1], -1), (1, 0))            # decay up to each chunk's start
    far = torch.ones(nc + 1, nc, dtype=torch.bool, device=x.device).tril(-1)
    carry = torch.exp(torch.where(far, total[..., :, None] - total[..., None, 1:], -torch.inf)).float()
    states = torch.matmul(carry, local.flatten(-2)).unflatten(-1, local.shape[-2:])
    if state is not None:
        states = states + torch.exp(total).float()[..., None, None] * state[:, :, None]
    y = y + torch.exp(cum).float()[..., None] * torch.matmul(ch, states[:, :, :-1])
    if D is not None:
        y = y + D[None, :, None, None, None] * xc
    y = y.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :L]
    return _packed(y, cu, T), states[:, :, -1]


def _plain_norm(x, residual, weight):
    """(y, h): h = x + residual in the residual's type, y its norm in 32 bits."""
    h = x.float()
    if residual is not None:
        h = (h + residual.float()).to(residual.dtype).float()
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * weight.float(), h


def _quantise(y, kind, group):
    rows, D = y.shape
    width = D if group == 0 else group
    top = FP8_MAX if kind == "fp8" else INT8_MAX
    yg = F.pad(y, (0, (-D) % width)).unflatten(1, (-1, width))
    scale = (yg.abs().amax(-1) / top).clamp_min(TINY)
    q = (yg / scale[..., None]).clamp(-top, top).flatten(1)[:, :D]
    if kind == "fp8":
        return q.to(torch.float8_e4m3fn), scale
    return torch.round(q).to(torch.int8), scale


def _stand_for(q, scale, group, dtype):
    """The values an int8 row stands for."""
    D = q.shape[1]
    s = scale if group == 0 else scale.repeat_interleave(group, dim=1)[:, :D]
    return (q.float() * s).to(dtype)


def _plain(s):
    case, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    f = lambda t: None if t is None else t.float()  # noqa: E731
    if case["mode"] != "train":
        if case["op"] == "norm":
            y, h = _plain_norm(s["x"], s["residual"], s["weight"])
            out = {} if s["residual"] is None else {"h": h.to(s["residual"].dtype)}
            if case["mode"] == "fwd":
                return {"y": y.to(dtype), **out}
            q, scale = _quantise(y, case["quant"], case["group"])
            if case["quant"] == "int8":
                q = _stand_for(q, scale, case["group"], dtype)
            return {"q": q, "scale": scale, **out}
        if case["op"] == "conv":
            y, last = _plain_conv(f(s["x"]), f(s["weight"]), f(s["bias"]), f(s["state"]),
                                  case["silu"], s["cu"], s["cu_cpu"])
            last = last.to(dtype)
        else:
            y, last = _plain_scan(f(s["x"]), s["dt"], s["A_log"], f(s["B"]), f(s["C"]), f(s["D"]),
                                  s["dt_bias"], s["state"], s["cu"], s["cu_cpu"])
        if case["mode"] == "step":          # the cache is updated in place
            s["state"].copy_(last)
            last = s["state"]
        return {"y": y.to(dtype), "state": last}

    with torch.enable_grad():
        if case["op"] == "norm":
            y, h = _plain_norm(s["x"], s["residual"], s["weight"])
            outs, grads = [y.to(dtype)], [s["dy"]]
            if s["residual"] is not None:
                outs.append(h.to(s["residual"].dtype))
                grads.append(s["dres"])
        else:
            if case["op"] == "conv":
                y, last = _plain_conv(f(s["x"]), f(s["weight"]), f(s["bias"]), f(s["state"]),
                                      case["silu"], s["cu"], s["cu_cpu"])
                last = last.to(dtype)
            else:
                y, last = _plain_scan(f(s["x"]), s["dt"], s["A_log"], f(s["B"]), f(s["C"]),
                                      f(s["D"]), s["dt_bias"], s["state"], s["cu"], s["cu_cpu"])
            outs, grads = [y.to(dtype)], [s["dy"]]
            if s["dstate"] is not None:
                outs.append(last)
                grads.append(s["dstate"])
        got = torch.autograd.grad(outs, s["leaves"], grads)
    return {"out": [o.detach() for o in outs], "grad": list(got)}


# ---- the framework's calls ------------------------------------------------------

def _own(s):
    import gated_delta_rule_66_amd as gdr
    case = s["case"]
    if case["op"] == "norm":
        if case["mode"] == "quant":
            q, scale, h = gdr.rms_norm_quant(s["x"], s["weight"], EPS, residual=s["residual"],
                                             format=case["quant"], group_size=case["group"])
            if case["quant"] == "int8":
                q = _stand_for(q, scale, case["group"], s["x"].dtype)
            return {"q": q, "scale": scale, **({} if h is None else {"h": h})}
        out = gdr.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
        outs = [out] if s["residual"] is None else list(out)
        if case["mode"] == "fwd":
            return dict(zip(("y", "h"), outs))
        grads = [s["dy"], s["dres"]][:len(outs)]
    else:
        seq = dict(initial_state=s["state"], cu_seqlens=s["cu"], cu_seqlens_cpu=s["cu_cpu"])
        if case["op"] == "conv":
            if case["mode"] == "step":
                y = gdr.causal_conv1d_update(s["x"], s["state"], s["weight"], s["bias"],
                                             activation=s["activation"])
                return {"y": y, "state": s["state"]}
            y, last = gdr.causal_conv1d(s["x"], s["weight"], s["bias"], activation=s["activation"],
                                        output_final_state=case["mode"] == "fwd" or case["state"],
                                        **seq)
        else:
            args = (s["x"], s["dt"], s["A_log"], s["B"], s["C"])
            kw = dict(D=s["D"], dt_bias=s["dt_bias"])
            if case["mode"] == "step":
                y, last = gdr.fused_recurrent_selective_scan(*args, **kw, initial_state=s["state"],
                                                             inplace_final_state=True)
                return {"y": y, "state": last}
            y, last = gdr.chunk_selective_scan(
                *args, **kw, output_final_state=case["mode"] == "fwd" or case["state"], **seq)
        if case["mode"] == "fwd":
            return {"y": y, "state": last}
        outs, grads = [y], [s["dy"]]
        if s["dstate"] is not None:
            outs.append(last)
            grads.append(s["dstate"])
    got = torch.autograd.grad(outs, s["leaves"], grads)
    return {"out": [o.detach() for o in outs], "grad": list(got)}


def run(state):
    if own:
        return _own(state)
    if state["case"]["mode"] == "train":
        return _plain(state)
    with torch.no_grad():
        return _plain(state)


# ---- what a pass has to move and compute ------------------------------------------

def work(case):
    es = DTYPES[case["dtype"]].itemsize
    train = case["mode"] == "train"
    if case["op"] == "norm":
        rows, D = case["rows"], case["D"]
        rs = {"none": 0, "same": es, "fp32": 4}[case["residual"]]
        out = 1 if case["quant"] else es
        byt = rows * D * (es + 2 * rs + out) + D * es       # x, residual in and out, y, weight
        if case["quant"]:
            byt += 4 * rows * (1 if case["group"] == 0 else -(-D // case["group"]))
        flops = 4 * rows * D
        if train:                                          # dy, its residual's, h again; dx, dresidual
            byt += rows * D * (es + rs + (rs or es) + es + rs) + D * es
            flops += 10 * rows * D
        return {"bytes": byt, "flops": flops}
    lens = _lens_of(case)
    n_seq = case["B"] if lens is None else len(lens)
    tok = case["B"] * case["T"]
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        st = n_seq * (W - 1) * D * es
        byt = tok * D * 2 * es + D * (W + 1) * es + st * (2 if case["state"] else 1)
        flops = tok * D * (2 * W + 4)
        if train:                                          # x and dy read, dx written
            byt += tok * D * 3 * es + D * (W + 1) * es + (2 * st if case["state"] else 0)
            flops += tok * D * (6 * W + 8)
        return {"bytes": byt, "flops": flops}
    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    st = n_seq * H * N * P * 4
    byt = tok * (2 * H * P + H + 2 * G * N) * es + (2 if case["state"] else 1) * st
    # per token and head: B x^T into the state, C S out of it
    flops = tok * H * (4 * N * P + 2 * N * P)
    if train:                                              # all inputs and dy read, all gradients written
        byt += tok * (3 * H * P + 2 * H + 4 * G * N) * es + 2 * st
        flops += tok * H * 12 * N * P
    return {"bytes": byt, "flops": flops}


# ---- the definitions in 64 bits ----------------------------------------------------

def _d(t):
    return None if t is None else t.detach().double()


def _spans(s):
    """(row, first token, last token + 1, sequence) of every sequence."""
    if s["cu_cpu"] is None:
        return [(b, 0, s["x"].shape[1], b) for b in range(s["x"].shape[0])]
    cu = s["cu_cpu"].tolist()
    return [(0, a, b, n) for n, (a, b) in enumerate(zip(cu, cu[1:]))]


def _exact_conv(s):
    case = s["case"]
    x, w, bias, st = (_d(s[k]) for k in ("x", "weight", "bias", "state"))
    W = case["W"]
    train = case["mode"] == "train"
    dy = _d(s["dy"]) if train else None
    dst = _d(s["dstate"]) if train else None
    y, last, dx = torch.empty_like(x), [], torch.empty_like(x)
    dw, db, dh = torch.zeros_like(w), torch.zeros_like(w[:, 0]), []
    for row, a, b, n in _spans(s):
        head = x.new_zeros(W - 1, x.shape[2]) if st is None else st[n]
        ext = torch.cat([head, x[row, a:b]])
        z = sum(ext[j:j + b - a] * w[:, j] for j in range(W))
        if bias is not None:
            z = z + bias
        sig = 1 / (1 + torch.exp(-z))
        y[row, a:b] = z * sig if case["silu"] else z
        last.append(ext[b - a:])
        if train:
            dz = dy[row, a:b] * (sig * (1 + z * (1 - sig)) if case["silu"] else 1.0)
            dext = torch.zeros_like(ext)
            for j in range(W):
                dext[j:j + b - a] += dz * w[:, j]
                dw[:, j] += (dz * ext[j:j + b - a]).sum(0)
            db += dz.sum(0)
            if dst is not None:
                dext[b - a:] += dst[n]
            dx[row, a:b] = dext[W - 1:]
            dh.append(dext[:W - 1])
    if not train:
        return {"y": y, "state": torch.stack(last)}
    outs = [y] + ([torch.stack(last)] if dst is not None else [])
    grads = [dx, dw] + ([db] if bias is not None else []) + ([torch.stack(dh)] if st is not None else [])
    return {"out": outs, "grad": grads}


def _exact_scan(s):
    """Token by token, all sequences at once (a sequence that has ended gets
    steps of size zero); the reverse pass recomputes the states of 64 tokens
    at a time from a kept one."""
    case = s["case"]
    x, raw, al, Bm, Cm, D, bias, h0 = (_d(s[k]) for k in ("x", "dt", "A_log", "B", "C", "D", "dt_bias",
                                                          "state"))
    spans = _spans(s)
    R = case["H"] // case["G"]
    n, L = len(spans), max(b - a for _, a, b, _ in spans)

    def gather(v):
        out = v.new_zeros((n, L) + v.shape[2:])
        for row, a, b, i in spans:
            out[i, :b - a] = v[row, a:b]
        return out

    def spread(v):
        out = v.new_zeros((case["B"], case["T"]) + v.shape[2:])
        for row, a, b, i in spans:
            out[row, a:b] = v[i, :b - a]
        return out

    z = raw + bias
    step = gather(torch.where(z > 30, z, torch.log1p(torch.exp(z))))
    rate = -torch.exp(al)
    xs, bs, cs = gather(x), gather(Bm), gather(Cm)
    S = x.new_zeros(n, case["H"], case["N"], case["P"]) if h0 is None else h0.clone()
    y = torch.zeros_like(xs)
    every = 64
    kept = []
    train = case["mode"] == "train"

    def forward(S, t):
        b = bs[:, t].repeat_interleave(R, 1)
        a = torch.exp(rate * step[:, t])[..., None, None]
        return a * S + (step[:, t, :, None] * b)[..., :, None] * xs[:, t][..., None, :]

    for t in range(L):
        if train and t % every == 0:
            kept.append(S)
        S = forward(S, t)
        c = cs[:, t].repeat_interleave(R, 1)
        y[:, t] = (c[..., :, None] * S).sum(-2)
    if D is not None:
        y = y + D[:, None] * xs
    if not train:
        return {"y": spread(y), "state": S}

    dy = gather(_d(s["dy"]))
    dS = torch.zeros_like(S) if s["dstate"] is None else _d(s["dstate"]).clone()
    dx = torch.zeros_like(xs) if D is None else D[:, None] * dy
    dstep, db, dc = torch.zeros_like(step), torch.zeros_like(bs), torch.zeros_like(cs)
    drate = torch.zeros_like(rate)
    groups = lambda v: v.unflatten(1, (case["G"], R)).sum(2)  # noqa: E731
    for t0 in reversed(range(0, L, every)):
        states = [kept.pop()]
        for t in range(t0, min(L, t0 + every)):
            states.append(forward(states[-1], t))
        for t in reversed(range(t0, min(L, t0 + every))):
            b, c = (v[:, t].repeat_interleave(R, 1) for v in (bs, cs))
            dc[:, t] = groups((states[t - t0 + 1] * dy[:, t][..., None, :]).sum(-1))
            dS = dS + c[..., :, None] * dy[:, t][..., None, :]
            sx = (dS * xs[:, t][..., None, :]).sum(-1)                # [n, H, N]
            db[:, t] = groups(step[:, t, :, None] * sx)
            dx[:, t] += step[:, t, :, None] * (dS * b[..., :, None]).sum(-2)
            a = torch.exp(rate * step[:, t])
            da = (dS * states[t - t0]).sum((-1, -2)) * a              # gradient of the log decay
            dstep[:, t] = (b * sx).sum(-1) + rate * da
            drate += (step[:, t] * da).sum(0)
            dS = a[..., None, None] * dS
    draw_ = spread(dstep) / (1 + torch.exp(-z))
    grads = [spread(dx), draw_, drate * rate, spread(db), spread(dc)]
    if D is not None:
        grads.append((_d(s["dy"]) * x).sum((0, 1, 3)))
    grads.append(draw_.sum((0, 1)))
    if h0 is not None:
        grads.append(dS)
    return {"out": [spread(y)] + ([S] if s["dstate"] is not None else []), "grad": grads}


def _exact_norm(s):
    case = s["case"]
    x, res, w = (_d(s[k]) for k in ("x", "residual", "weight"))
    h = x
    if res is not None:  # the stored stream is what is normalised: its rounding is part of the definition
        h = (s["x"].detach().float() + s["residual"].detach().float()).to(s["residual"].dtype).double()
    inv = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    unit = h * inv
    y = unit * w
    if case["mode"] == "quant":
        top = FP8_MAX if case["quant"] == "fp8" else INT8_MAX
        width = case["group"] or case["D"]
        yg = F.pad(y, (0, (-case["D"]) % width)).unflatten(1, (-1, width))
        scale = (yg.abs().amax(-1) / top).clamp_min(TINY)
        q = yg / scale[..., None]
        if case["quant"] == "int8":
            q = torch.round(q) * scale[..., None]
        # an fp8 value is held against what it was rounded from
        out = {"q": q.flatten(1)[:, :case["D"]], "scale": scale}
        return out if res is None else {**out, "h": h}
    if case["mode"] == "fwd":
        return {"y": y} if res is None else {"y": y, "h": h}
    dy = _d(s["dy"])
    du = dy * w
    dh = inv * (du - unit * (du * unit).mean(-1, keepdim=True))
    if res is not None:
        dh = dh + _d(s["dres"])
    grads = [dh] + ([dh] if res is not None else []) + [(dy * unit).sum(0)]
    return {"out": [y] + ([h] if res is not None else []), "grad": grads}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "conv":
            return _exact_conv(s)
        if case["op"] == "norm":
            return _exact_norm(s)
        return _exact_scan(s)
