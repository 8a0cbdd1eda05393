"""The block operators around the scan, as cases to be measured.

Four operators: the gated linear recurrence (`gated_scan`, its single-token
step and its backward pass), the residual norm in front of a block
(`add_rms_norm`), the gated norm behind the recurrence (`gated_rms_norm`), each
with its backward pass, and the backward pass of `causal_conv1d`.

A case says its sequences by `lens` (a text of token counts; they are packed
into one stream with offsets, or a dense batch of equal lengths where `dense`
is true).  `run` computes a case in elementary torch operations in fp32, or,
where `own` is true, by the package's own calls.
"""
import math

import torch

own = False

RATE = 8.0   # a = exp(-RATE softplus(lam) sigmoid(r))
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token through a small layer: launch latency
        {"name": "step-one", "op": "step", "rows": 1, "channels": 1536, "dtype": "bf16"},
        # a full serving batch at the 2.7B-shaped inner width
        {"name": "step-batch", "op": "step", "rows": 256, "channels": 5120, "dtype": "bf16"},
        # one prompt of the 130M-shaped workload: few channels, the work split over the tokens
        {"name": "scan-prompt", "op": "scan", "lens": "4096", "dense": True, "channels": 1536, "dtype": "bf16"},
        # the packed prefill: four prompts of very different lengths, 128 heads of 64 channels
        {"name": "scan-packed", "op": "scan", "lens": "1024,4096,12288,32768", "dense": False, "channels": 8192,
         "dtype": "bf16"},
        # a training step of the recurrence: forward and backward at the 2.7B-shaped model width
        {"name": "scan-train", "op": "scan-train", "lens": ",".join(["8192"] * 8), "dense": True, "channels": 2560,
         "dtype": "bf16"},
        # fp32 training on documents packed without padding, one of them empty, one a single token
        {"name": "scan-train-ragged", "op": "scan-train", "lens": "1,700,0,2049,333,5000", "dense": False,
         "channels": 776, "dtype": "f32"},
        # a decode step's norm in front of the next block
        {"name": "residual-decode", "op": "residual", "rows": 256, "channels": 2560, "dtype": "bf16",
         "residual": "bf16", "scaled": True},
        # forward and backward over a training batch, the residual stream kept in fp32
        {"name": "residual-train", "op": "residual-train", "rows": 65536, "channels": 2560, "dtype": "bf16",
         "residual": "f32", "scaled": True},
        # a decode step's norm behind the scan, whose output is fp32 by default
        {"name": "gate-decode", "op": "gate", "rows": 256, "channels": 5120, "dtype": "bf16", "input": "f32",
         "groups": 1, "norm_first": False},
        # forward and backward over the packed workload's tokens, one norm per B/C group
        {"name": "gate-train", "op": "gate-train", "rows": 49152, "channels": 8192, "dtype": "bf16", "input": "bf16",
         "groups": 8, "norm_first": False},
        # the convolution's gradients at the 2.7B-shaped xBC width, its outputs' gradients in three parts
        {"name": "conv-train", "op": "conv", "lens": ",".join(["8192"] * 8), "dense": True, "channels": 5376,
         "width": 4, "silu": True, "dtype": "bf16", "parts": "5120,128,128"},
        # fp32 gradients over packed documents shorter than the window and over many blocks, with states
        {"name": "conv-train-ragged", "op": "conv", "lens": "1,700,0,2049,333,5000", "dense": False, "channels": 136,
         "width": 3, "silu": True, "dtype": "f32", "parts": "136"},
    ]


def _between(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(rng, most):
    """Token counts of a batch of at most `most` tokens: equal ones, or a ragged packed list."""
    total = _between(rng, 16, most)
    if rng.random() < 0.5:
        b = min(_between(rng, 1, 64), total)
        return ",".join([str(total // b)] * b), True
    n = min(_between(rng, 1, 32), total)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(hi - lo) for lo, hi in zip([0] + cuts, cuts + [total])), False


def draw(rng):
    op = rng.choice(["step", "scan", "scan-train", "residual", "residual-train", "residual-backward", "gate",
                     "gate-train", "conv"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    channels = 8 * _between(rng, 8, 1024)
    case = {"op": op, "channels": channels, "dtype": dtype}
    most = min(65536, (1 << 27) // channels)
    if op in ("scan", "scan-train", "conv"):
        case["lens"], case["dense"] = _lens(rng, most)
    else:
        case["rows"] = _between(rng, 1, 2048 if op == "step" else most)
    if op.startswith("residual"):
        case["residual"] = "f32" if op == "residual-train" else rng.choice([dtype, "f32"])
        case["scaled"] = rng.random() < 0.5
    if op.startswith("gate"):
        case["input"] = rng.choice([dtype, "f32"])
        case["groups"] = rng.choice([g for g in (1, 1, 2, 4, 8) if channels % (8 * g) == 0])
        case["norm_first"] = rng.random() < 0.5
    if op == "conv":
        case["width"] = rng.choice([2, 3, 4, 4])
        case["silu"] = rng.random() < 0.75
        p = 8 * rng.randint(0, channels // 8 - 1)
        case["parts"] = "%d,%d" % (p, channels - p) if p else str(channels)
    return case


def work(case):
    """Bytes and operations of one pass, each input read once and each output written once."""
    op, C, e = case["op"], case["channels"], TYPES[case["dtype"]].itemsize
    if "lens" in case:
        lens = [int(n) for n in case["lens"].split(",")]
        rows, states = sum(lens), len(lens) * C
    else:
        rows = case["rows"]
    n = rows * C
    if op == "step":
        return {"bytes": n * (4 * e + 8) + 4 * C, "flops": 25 * n}
    if op == "scan":  # x, r, i in, y out; initial and final states
        return {"bytes": n * 4 * e + 8 * states + 4 * C, "flops": 25 * n}
    if op == "scan-train":  # the forward, then x, r, i, dy in and dx, dr, di out, and the states' gradients
        return {"bytes": n * 11 * e + 16 * states + 8 * C, "flops": 80 * n}
    if op in ("residual", "residual-train", "residual-backward"):
        u, s = TYPES[case["residual"]].itemsize, 4 * C if case["scaled"] else 0
        forward = n * (2 * e + 2 * u) + 4 * C + s + 4 * rows  # x, residual in, y, residual out
        # dy, the later residual's gradient, the residual (and x for the scale's gradient) in; dx, dresidual out
        backward = n * ((3 if s else 2) * e + 3 * u) + 8 * C + 2 * s + 4 * rows
        parts = (op != "residual-backward") * forward + (op != "residual") * backward
        return {"bytes": parts, "flops": n * (6 * (op != "residual-backward") + 14 * (op != "residual"))}
    if op in ("gate", "gate-train"):
        i = TYPES[case["input"]].itemsize
        forward = n * (i + 2 * e) + 4 * C + 4 * rows * case["groups"]  # x, z in, y out
        backward = n * (2 * i + 3 * e) + 8 * C + 4 * rows * case["groups"]  # dy, x, z in, dx, dz out
        return {"bytes": forward + (op == "gate-train") * backward, "flops": n * (10 + 30 * (op == "gate-train"))}
    K = case["width"]  # conv: x, dy in, dx out; weights, bias and states with their gradients
    return {"bytes": n * 3 * e + 8 * C * (K + 1) + 3 * e * states * (K - 1), "flops": n * (6 * K + 12)}


# ------------------------------------------------------------------ inputs
class _Draws:
    """Normal and uniform values on the GPU from one seed."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0, add=0.0):
        v = torch.randn(shape, generator=self.g, device="cuda")
        if scale != 1.0:
            v *= scale
        if add:
            v += add
        return v.to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(shape, generator=self.g, device="cuda") * (hi - lo) + lo


def _decay(d, C):
    """lam such that exp(-RATE softplus(lam)) is spread over (0.9, 0.999): memories of ten to a thousand tokens."""
    a = d.uniform(0.9, 0.999, C).double()
    return torch.log(torch.expm1(-torch.log(a) / RATE)).float()


def _sequences(case):
    """The offsets as the calls take them, and for the plain form the place of each token in its sequence."""
    lens = [int(n) for n in case["lens"].split(",")]
    counts = torch.tensor(lens, dtype=torch.int64)
    cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
    cu[1:] = counts.cumsum(0)
    seq = torch.repeat_interleave(torch.arange(len(lens)), counts)
    pos = torch.arange(int(cu[-1])) - cu[seq]
    full = (counts > 0).nonzero()[:, 0]
    plan = {"lens": lens, "T": int(cu[-1]), "cu": cu.to(torch.int32), "seq": seq, "pos": pos, "left": counts[seq] - 1 - pos,
            "full": full, "first": cu[full], "last": cu[full + 1] - 1, "counts": counts}
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in plan.items()}


def prepare(case, seed):
    d, C, t = _Draws(seed), case["channels"], TYPES[case["dtype"]]
    op, s = case["op"], {"case": dict(case)}
    if op == "step":
        n = case["rows"]
        s |= {"lam": _decay(d, C), "state": d.normal(n, C)}
        s |= {k: d.normal(n, C, dtype=t) for k in ("x", "r", "i")}
        s["after"] = torch.empty_like(s["state"])
        s["y"] = torch.empty_like(s["x"])
        return s
    if op in ("scan", "scan-train"):
        s["plan"] = p = _sequences(case)
        n = len(p["lens"])
        lead = (n, p["lens"][0]) if case["dense"] else (p["T"],)
        s |= {"lam": _decay(d, C), "init": d.normal(n, C)}
        s |= {k: d.normal(*lead, C, dtype=t) for k in ("x", "r", "i")}
        if op == "scan-train":
            s |= {"dy": d.normal(*lead, C, dtype=t), "dfinal": d.normal(n, C)}
        return s
    if op == "conv":
        s["plan"] = p = _sequences(case)
        n, K = len(p["lens"]), case["width"]
        lead = (n, p["lens"][0]) if case["dense"] else (p["T"],)
        s["parts"] = [int(c) for c in case["parts"].split(",")]
        s |= {"x": d.normal(*lead, C, dtype=t), "weight": d.normal(C, K, scale=K ** -0.5),
              "bias": d.normal(C, scale=0.1), "state": d.normal(n, K - 1, C, dtype=t),
              "dfinal": d.normal(n, K - 1, C, dtype=t), "dys": [d.normal(*lead, c, dtype=t) for c in s["parts"]]}
        # the tokens whose window reaches into the incoming state, by how far back the tap lies
        s["head"] = [None] + [(p["pos"] < k).nonzero()[:, 0] for k in range(1, K)]
        # of each sequence's last inputs (its outgoing state), those that are tokens and those of the incoming state
        j = torch.arange(K - 1, device="cuda")[None, :]
        at = p["counts"][:, None] + j
        s["tail_token"] = (at >= K - 1).nonzero()
        s["tail_state"] = (at < K - 1).nonzero()
        return s
    n = case["rows"]
    s["weight"] = d.normal(C, scale=0.1, add=1.0)
    if op.startswith("residual"):
        u = TYPES[case["residual"]]
        s["scale"] = d.uniform(0.1, 1.0, C) if case["scaled"] else None
        s["x"] = d.normal(n, C, dtype=t)
        if op != "residual-backward":
            s["residual"] = d.normal(n, C, dtype=u, scale=2.0)
        if op != "residual":
            s |= {"dy": d.normal(n, C, dtype=t), "dout": d.normal(n, C, dtype=u)}
        if op == "residual-backward":  # what the forward pass left behind
            s["out"] = d.normal(n, C, dtype=u, scale=2.0)
            s["rstd"] = torch.rsqrt(s["out"].float().square().mean(-1) + EPS)
        return s
    s |= {"x": d.normal(n, C, dtype=TYPES[case["input"]], scale=0.5), "z": d.normal(n, C, dtype=t)}
    if op == "gate-train":
        s["dy"] = d.normal(n, C, dtype=t)
    return s


# ------------------------------------------------------------------ plain forms
def _doubling(a, b):
    """h[:, t] = a[:, t] h[:, t-1] + b[:, t] along dim 1 with h before it zero, and the running products of a."""
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return a, b


def _recurrence(a, b, block=32):
    """h_t = a_t h_{t-1} + b_t over dim 0 of [T, C], h_{-1} = 0: doubling in blocks, then over the blocks."""
    T, C = a.shape
    pad = -T % block
    if pad:
        a = torch.cat([a, a.new_zeros(pad, C)])
        b = torch.cat([b, b.new_zeros(pad, C)])
    a, b = _doubling(a.view(-1, block, C), b.view(-1, block, C))
    _, h = _doubling(a[None, :, -1], b[None, :, -1])
    before = torch.cat([h.new_zeros(1, C), h[0, :-1]])
    return (b + a * before[:, None]).view(-1, C)[:T]


def _gates(x, r, i, lam):
    loga = -RATE * torch.nn.functional.softplus(lam) * torch.sigmoid(r)
    beta = torch.sqrt(-torch.expm1(2 * loga))
    return loga, torch.exp(loga), beta, torch.sigmoid(i)


def _flat(s, *names):
    return [s[n].float().reshape(-1, s[n].shape[-1]) for n in names]


def _scan_plain(s, p):
    """Every h [T, C], the final states, and what the backward pass needs."""
    x, r, i = _flat(s, "x", "r", "i")
    loga, a, beta, gate = _gates(x, r, i, s["lam"])
    b = beta * gate * x
    b[p["first"]] += a[p["first"]] * s["init"][p["full"]]
    inside = a.clone()
    inside[p["first"]] = 0
    h = _recurrence(inside, b)
    final = s["init"].clone()
    final[p["full"]] = h[p["last"]]
    return h, final, (x, r, loga, a, beta, gate, inside)


def _scan_backward_plain(s, p, h, kept):
    x, r, loga, a, beta, gate, inside = kept
    (dy,) = _flat(s, "dy")
    dy = dy.clone()
    dy[p["last"]] += s["dfinal"][p["full"]]
    # g_t = dy_t + a_{t+1} g_{t+1}, run from the end
    after = torch.cat([inside[1:], inside.new_zeros(1, inside.shape[1])])
    g = _recurrence(after.flip(0), dy.flip(0)).flip(0)
    dinit = s["dfinal"].clone()
    dinit[p["full"]] = a[p["first"]] * g[p["first"]]
    before = torch.cat([h.new_zeros(1, h.shape[1]), h[:-1]])
    before[p["first"]] = s["init"][p["full"]]
    dx = g * beta * gate
    di = g * beta * x * gate * (1 - gate)
    # d beta / d loga = -a^2 / beta; where loga is 0 the product with it is 0
    dloga = g * (a * before - torch.where(beta > 0, a * a / beta, 0.0) * gate * x) * loga
    dr = dloga * (1 - torch.sigmoid(r))
    dlam = dloga.sum(0) * torch.sigmoid(s["lam"]) / torch.nn.functional.softplus(s["lam"])
    return dx, dr, di, dlam, dinit


def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    g = torch.sigmoid(v)
    return g * (1 + v * (1 - g))


def _residual_plain(s):
    x, u = s["x"].float(), s["residual"].float()
    u = u + (x if s["scale"] is None else s["scale"] * x)
    rstd = torch.rsqrt(u.square().mean(-1) + EPS)
    return (u * rstd[:, None] * s["weight"]).to(s["x"].dtype), u.to(s["residual"].dtype), rstd


def _residual_backward_plain(s, out, rstd):
    dy, u = s["dy"].float(), out.float() * rstd[:, None]
    wdy = dy * s["weight"]
    dres = s["dout"].float() + rstd[:, None] * (wdy - u * (wdy * u).mean(-1, keepdim=True))
    dx = dres if s["scale"] is None else dres * s["scale"]
    dscale = None if s["scale"] is None else (dres * s["x"].float()).sum(0)
    return dx.to(s["x"].dtype), dres.to(out.dtype), (dy * u).sum(0), dscale


def _gate_plain(s, groups, norm_first):
    x, z = s["x"].float(), s["z"].float()
    n, C = x.shape
    v = x if norm_first else x * _silu(z)
    v = v.view(n, groups, C // groups)
    rstd = torch.rsqrt(v.square().mean(-1) + EPS)
    y = (v * rstd[:, :, None]).view(n, C) * s["weight"]
    if norm_first:
        y = y * _silu(z)
    return y.to(s["z"].dtype), rstd


def _gate_backward_plain(s, rstd, groups, norm_first):
    x, z, dy = s["x"].float(), s["z"].float(), s["dy"].float()
    n, C = x.shape
    gate = _silu(z)
    v = x if norm_first else x * gate
    u = (v.view(n, groups, -1) * rstd[:, :, None]).view(n, C)
    dn = dy * gate if norm_first else dy
    dweight = (dn * u).sum(0)
    wd = dn * s["weight"]
    mean = (wd * u).view(n, groups, -1).mean(-1, keepdim=True)
    dv = (rstd[:, :, None] * (wd.view(n, groups, -1) - u.view(n, groups, -1) * mean)).view(n, C)
    if norm_first:
        dx, dgate = dv, dy * u * s["weight"]
    else:
        dx, dgate = dv * gate, dv * x
    return dx.to(s["x"].dtype), (dgate * _dsilu(z)).to(s["z"].dtype), dweight


def _conv_plain(s, p, K, silu):
    (x,) = _flat(s, "x")
    dy = torch.cat([v.float().reshape(-1, v.shape[-1]) for v in s["dys"]], 1)
    w, st = s["weight"], s["state"].float()
    C = x.shape[1]

    def earlier(k):
        """The input k tokens before each token: of its sequence, or of the state before it."""
        if not k:
            return x
        v = torch.cat([x.new_zeros(min(k, len(x)), C), x[:-k]])
        rows = s["head"][k]
        v[rows] = st[p["seq"][rows], p["pos"][rows] + K - 1 - k]
        return v

    taps = [earlier(K - 1 - k) for k in range(K)]
    v = sum(w[:, k] * taps[k] for k in range(K)) + s["bias"]
    dv = dy * _dsilu(v) if silu else dy
    dweight = torch.stack([(dv * taps[k]).sum(0) for k in range(K)], 1)

    def later(k):
        """dv of the token k after each token of the same sequence, 0 behind its end."""
        return dv if not k else torch.where((p["left"] >= k)[:, None], torch.cat([dv[k:], dv.new_zeros(min(k, len(dv)), C)]), 0.0)

    dx = sum(w[:, k] * later(K - 1 - k) for k in range(K))
    dstate = torch.zeros_like(st)
    for k in range(K - 1):
        rows = s["head"][K - 1 - k]
        dstate[p["seq"][rows], p["pos"][rows] + k] += w[:, k] * dv[rows]
    q, j = s["tail_token"].unbind(1)
    dx[p["cu"][q + 1].long() + j - (K - 1)] += s["dfinal"][q, j].float()
    q, j = s["tail_state"].unbind(1)
    dstate[q, p["counts"][q] + j] += s["dfinal"][q, j].float()
    return dx.to(s["x"].dtype).view_as(s["x"]), dweight, dv.sum(0), dstate.to(s["x"].dtype)


def _run_plain(s):
    case = s["case"]
    op, t = case["op"], TYPES[case["dtype"]]
    if op == "step":
        x, r, i = _flat(s, "x", "r", "i")
        _, a, beta, gate = _gates(x, r, i, s["lam"])
        h = a * s["state"] + beta * gate * x
        return {"y": h.to(t), "state": h}
    if op == "scan":
        h, final, _ = _scan_plain(s, s["plan"])
        return {"y": h.to(t).view_as(s["x"]), "final": final}
    if op == "scan-train":
        h, final, kept = _scan_plain(s, s["plan"])
        dx, dr, di, dlam, dinit = _scan_backward_plain(s, s["plan"], h, kept)
        return {"y": h.to(t).view_as(s["x"]), "final": final, "dx": dx.to(t).view_as(s["x"]),
                "dr": dr.to(t).view_as(s["x"]), "di": di.to(t).view_as(s["x"]), "dlam": dlam, "dinit": dinit}
    if op == "residual":
        y, out, _ = _residual_plain(s)
        return {"y": y, "out": out}
    if op == "residual-train":
        y, out, rstd = _residual_plain(s)
        dx, dres, dweight, dscale = _residual_backward_plain(s, out, rstd)
        return {"y": y, "out": out, "dx": dx, "dresidual": dres, "dweight": dweight, "dscale": dscale}
    if op == "residual-backward":
        dx, dres, dweight, dscale = _residual_backward_plain(s, s["out"], s["rstd"])
        return {"dx": dx, "dresidual": dres, "dweight": dweight, "dscale": dscale}
    if op == "gate":
        return {"y": _gate_plain(s, case["groups"], case["norm_first"])[0]}
    if op == "gate-train":
        y, rstd = _gate_plain(s, case["groups"], case["norm_first"])
        dx, dz, dweight = _gate_backward_plain(s, rstd, case["groups"], case["norm_first"])
        return {"y": y, "dx": dx, "dz": dz, "dweight": dweight}
    dx, dweight, dbias, dstate = _conv_plain(s, s["plan"], case["width"], case["silu"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dstate": dstate}


# ------------------------------------------------------------------ the package's calls
def _run_own(s):
    import mamba_ssd_chunked_02_amd as ssd
    case = s["case"]
    op, t = case["op"], TYPES[case["dtype"]]
    if op == "step":
        y = ssd.gated_scan_step(s["state"], s["x"], s["r"], s["i"], s["lam"], rate=RATE, state_out=s["after"], y=s["y"])
        return {"y": y, "state": s["after"]}
    if op in ("scan", "scan-train", "conv"):
        cu = None if case["dense"] else s["plan"]["cu"]
    if op == "scan":
        y, final = ssd.gated_scan(s["x"], s["r"], s["i"], s["lam"], rate=RATE, init_state=s["init"], cu_seqlens=cu)
        return {"y": y, "final": final}
    if op == "scan-train":
        y, final, states = ssd.gated_scan(s["x"], s["r"], s["i"], s["lam"], rate=RATE, init_state=s["init"],
                                          cu_seqlens=cu, want_states=True)
        dx, dr, di, dlam, dinit = ssd.gated_scan_backward(s["dy"], s["x"], s["r"], s["i"], s["lam"], states, rate=RATE,
                                                          init_state=s["init"], dfinal_state=s["dfinal"],
                                                          cu_seqlens=cu)
        return {"y": y, "final": final, "dx": dx, "dr": dr, "di": di, "dlam": dlam, "dinit": dinit}
    if op == "residual":
        y, out = ssd.add_rms_norm(s["x"], s["residual"], s["weight"], scale=s["scale"], eps=EPS)
        return {"y": y, "out": out}
    if op in ("residual-train", "residual-backward"):
        if op == "residual-train":
            y, out, rstd = ssd.add_rms_norm(s["x"], s["residual"], s["weight"], scale=s["scale"], eps=EPS, want_rstd=True)
        else:
            out, rstd = s["out"], s["rstd"]
        got = ssd.add_rms_norm_backward(s["dy"], out, s["weight"], rstd, dresidual_out=s["dout"],
                                        x=None if s["scale"] is None else s["x"], scale=s["scale"])
        got = dict(zip(("dx", "dresidual", "dweight", "dscale"), got))
        return got if op == "residual-backward" else {"y": y, "out": out, **got}
    if op in ("gate", "gate-train"):
        kind = {"groups": case["groups"], "norm_before_gate": case["norm_first"]}
        if op == "gate":
            return {"y": ssd.gated_rms_norm(s["x"], s["z"], s["weight"], eps=EPS, **kind)}
        y, rstd = ssd.gated_rms_norm(s["x"], s["z"], s["weight"], eps=EPS, want_rstd=True, **kind)
        dx, dz, dweight = ssd.gated_rms_norm_backward(s["dy"], s["x"], s["z"], s["weight"], rstd, **kind)
        return {"y": y, "dx": dx, "dz": dz, "dweight": dweight}
    dx, dweight, dbias, dstate = ssd.causal_conv1d_backward(s["dys"], s["x"], s["weight"], s["bias"], cu_seqlens=cu,
                                                            conv_state=s["state"], dfinal_conv_state=s["dfinal"],
                                                            activation=case["silu"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dstate": dstate}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ 64 bits
def _leaf(v):
    return v.double().requires_grad_()


def _exact_scan(s, case, train):
    """Token by token from the definition; gradients by differentiating it."""
    p = s["plan"]
    x, r, i = (_leaf(s[k].reshape(-1, case["channels"])) for k in ("x", "r", "i"))
    lam, init = _leaf(s["lam"]), _leaf(s["init"])
    leaves = (x, r, i, lam, init)
    with torch.set_grad_enabled(train):
        a = torch.exp(-RATE * torch.log1p(torch.exp(lam)) / (1 + torch.exp(-r)))
        b = torch.sqrt((1 - a) * (1 + a)) * x / (1 + torch.exp(-i))
        states, ys = list(init.unbind(0)), []
        bounds = [0] + torch.tensor(p["lens"]).cumsum(0).tolist()
        if case["dense"]:  # equal lengths: all sequences a token at a time
            n, L = len(p["lens"]), p["lens"][0]
            h, steps = init, []
            for at, bt in zip(a.view(n, L, -1).unbind(1), b.view(n, L, -1).unbind(1)):
                h = torch.addcmul(bt, at, h)
                steps.append(h)
            y, final = torch.stack(steps, 1).reshape(n * L, -1), h
        else:
            a, b = a.unbind(0), b.unbind(0)
            for q, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
                h = states[q]
                for t in range(lo, hi):
                    h = torch.addcmul(b[t], a[t], h)
                    ys.append(h)
                states[q] = h
            y, final = torch.stack(ys), torch.stack(states)
    got = {"y": y.detach().view(s["x"].shape), "final": final.detach()}
    if train:
        g = torch.autograd.grad([y, final], leaves, [s["dy"].double().reshape(y.shape), s["dfinal"].double()])
        got |= {k: v.view(s["x"].shape) for k, v in zip(("dx", "dr", "di"), g)}
        got |= {"dlam": g[3], "dinit": g[4]}
    return got


def _exact_norm(v, weight):
    return v / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS) * weight


def _exact_residual(s, op):
    w, x = _leaf(s["weight"]), _leaf(s["x"])
    scale = None if s["scale"] is None else _leaf(s["scale"])
    res = _leaf(s["out"]) if op == "residual-backward" else _leaf(s["residual"])
    if op == "residual-backward":  # `out` is given: the sum's value is out, its gradients flow to both terms
        s1 = torch.ones_like(w) if scale is None else scale
        with torch.no_grad():
            base = res - s1 * x
        res = base.requires_grad_()
    out = res + (x if scale is None else scale * x)
    y = _exact_norm(out, w)
    got = {} if op == "residual-backward" else {"y": y.detach(), "out": out.detach()}
    if op != "residual":
        leaves = [x, res, w] + ([] if scale is None else [scale])
        g = torch.autograd.grad([y, out], leaves, [s["dy"].double(), s["dout"].double()])
        got |= {"dx": g[0], "dresidual": g[1], "dweight": g[2], "dscale": g[3] if scale is not None else None}
    return got


def _exact_gate(s, case):
    x, z, w = _leaf(s["x"]), _leaf(s["z"]), _leaf(s["weight"])
    n, C = x.shape
    G = case["groups"]
    gate = z / (1 + torch.exp(-z))
    v = x if case["norm_first"] else x * gate
    y = _exact_norm(v.view(n, G, C // G), w.view(G, C // G)).reshape(n, C)
    if case["norm_first"]:
        y = y * gate
    got = {"y": y.detach()}
    if case["op"] == "gate-train":
        got |= dict(zip(("dx", "dz", "dweight"), torch.autograd.grad(y, [x, z, w], s["dy"].double())))
    return got


def _exact_conv(s, case):
    K, C = case["width"], case["channels"]
    x, w, b, st = _leaf(s["x"].reshape(-1, C)), _leaf(s["weight"]), _leaf(s["bias"]), _leaf(s["state"])
    dy = torch.cat([v.double().reshape(-1, v.shape[-1]) for v in s["dys"]], 1)
    outs, ends = [], []
    for q, part in enumerate(x.split(s["plan"]["lens"])):
        xp = torch.cat([st[q], part])
        v = b + sum(w[:, k] * xp[k:k + len(part)] for k in range(K))
        outs.append(v / (1 + torch.exp(-v)) if case["silu"] else v)
        ends.append(xp[len(part):])
    g = torch.autograd.grad([torch.cat(outs), torch.stack(ends)], [x, w, b, st], [dy, s["dfinal"].double()])
    return {"dx": g[0].view(s["x"].shape), "dweight": g[1], "dbias": g[2], "dstate": g[3]}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        with torch.no_grad():
            r, i, x = s["r"].double(), s["i"].double(), s["x"].double()
            a = torch.exp(-RATE * torch.log1p(torch.exp(s["lam"].double())) / (1 + torch.exp(-r)))
            h = a * s["state"].double() + torch.sqrt((1 - a) * (1 + a)) * x / (1 + torch.exp(-i))
        return {"y": h, "state": h}
    if op in ("scan", "scan-train"):
        return _exact_scan(s, case, op == "scan-train")
    if op.startswith("residual"):
        return _exact_residual(s, op)
    if op in ("gate", "gate-train"):
        return _exact_gate(s, case)
    return _exact_conv(s, case)
