"""The operators of a selective state space layer in their plain form, and the cases they are measured on.

What such a layer runs around its matrix products, for prompts and for single tokens:

* ``norm``  the residual's addition and the root-mean-square norm in front of a projection, with an
  output in 8 bits and its scales, or in 16 or 32,
* ``conv``  the causal convolution of width 4 with SiLU that its input passes, with the state it leaves,
* ``scan``  the state of every channel advanced over a prompt, with the readout of each position,
* ``step``  the same for the one new token of every request.

``run`` computes an operator with elementary torch operations where ``own`` is false, and with the
library's calls where it is true.
"""
import math

import torch

own = False

DEVICE = "cuda"
TOP = 448.0  # the largest value that 8 bits (e4m3) hold
EPS = 1e-6
LEAST = 1e-30  # scales are made as if the largest value were at least this


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # one user's token in front of a projection: latency
        {"name": "norm_one", "op": "norm", "rows": 1, "width": 2048, "x": "bf16", "residual": "bf16", "out": "bf16", "group": 0},
        # a full decode batch in front of an 8-bit projection, one scale a token
        {"name": "norm_step", "op": "norm", "rows": 256, "width": 4096, "x": "bf16", "residual": "bf16", "out": "e4m3", "group": 0},
        # packed prompts in front of an 8-bit projection with a scale for every 128 channels
        {"name": "norm_prompts", "op": "norm", "rows": 32749, "width": 4096, "x": "bf16", "residual": "bf16", "out": "e4m3", "group": 128},
        # the convolution of one decode step
        {"name": "conv_step", "op": "conv", "batch": 64, "T": 1, "channels": 6144, "x": "bf16", "ragged": False},
        # prompts of every length, admitted together
        {"name": "conv_prompts", "op": "conv", "batch": 8, "T": 4093, "channels": 4096, "x": "bf16", "ragged": True},
        # one user's prompt: the work has to be split along it
        {"name": "scan_one", "op": "scan", "batch": 1, "T": 1021, "channels": 2048, "state": 16, "groups": 1, "x": "bf16", "ragged": False, "gate": True},
        # a batch of prompts of every length
        {"name": "scan_prompts", "op": "scan", "batch": 8, "T": 2045, "channels": 4096, "state": 16, "groups": 1, "x": "bf16", "ragged": True, "gate": True},
        # one long document
        {"name": "scan_long", "op": "scan", "batch": 1, "T": 16384, "channels": 8192, "state": 16, "groups": 1, "x": "bf16", "ragged": False, "gate": True},
        # larger states in groups, fp32 inputs, no gate
        {"name": "scan_fp32", "op": "scan", "batch": 3, "T": 509, "channels": 2048, "state": 64, "groups": 4, "x": "fp32", "ragged": False, "gate": False},
        # one user's token
        {"name": "step_one", "op": "step", "batch": 1, "channels": 2048, "state": 16, "groups": 1, "x": "bf16", "gate": True},
        # a full decode batch
        {"name": "step_batch", "op": "step", "batch": 512, "channels": 4096, "state": 16, "groups": 1, "x": "bf16", "gate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "conv", "conv", "scan", "scan", "scan", "step", "step"])
    kind = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "norm":
        out = rng.choice(["e4m3", "e4m3", kind])
        while True:
            rows, width = _log(rng, 1, 32749), 8 * _log(rng, 8, 1024)
            if rows * width * (2 if kind == "fp32" else 1) <= 32749 * 4096 / 2:
                break
        return {"op": op, "rows": rows, "width": width, "x": kind, "residual": rng.choice([kind, kind, "fp32", "none"]), "out": out,
                "group": rng.choice([0, 128]) if out == "e4m3" else 0}
    channels = 8 * _log(rng, 8, 1024)
    if op == "conv":
        T = rng.choice([1, _log(rng, 2, 16384)])
        while True:
            batch = _log(rng, 1, 512)
            if batch * T * channels <= 8 * 4093 * 4096 / 2:
                break
            T, channels = max(1, T // 2), max(64, channels // 16 * 8)
        return {"op": op, "batch": batch, "T": T, "channels": channels, "x": kind, "ragged": T > 1 and rng.random() < 0.5}
    state, groups = rng.choice([8, 16, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
    channels = -(-channels // (8 * groups)) * 8 * groups
    if op == "step":
        while True:
            batch = _log(rng, 1, 512)
            if batch * channels * max(16, state) <= 512 * 4096 * 16:
                break
        return {"op": op, "batch": batch, "channels": channels, "state": state, "groups": groups, "x": kind, "gate": rng.random() < 0.7}
    while True:
        batch, T = _log(rng, 1, 64), _log(rng, 1, 16384)
        if batch * T * channels * max(16, state) * (2 if kind == "fp32" else 1) <= 16384 * 8192 * 16:
            break
    return {"op": op, "batch": batch, "T": T, "channels": channels, "state": state, "groups": groups, "x": kind,
            "ragged": rng.random() < 0.5, "gate": rng.random() < 0.7}


def _lengths(case):
    """The prompts' lengths, before a permutation: the same for every seed."""
    batch, T = case["batch"], case["T"]
    return [T - T * i // batch for i in range(batch)] if case.get("ragged") else [T] * batch


_SIZE = {"bf16": 2, "fp32": 4, "e4m3": 1, "none": 0}


def work(case):
    e = _SIZE[case["x"]]
    if case["op"] == "norm":
        n, d = case["rows"], case["width"]
        scales = (-(-d // case["group"]) if case["group"] else 1) if case["out"] == "e4m3" else 0
        return {"bytes": n * d * (e + 2 * _SIZE[case["residual"]] + _SIZE[case["out"]]) + n * scales * 4 + d * 4, "flops": 6 * n * d}
    D, B = case["channels"], case["batch"]
    tokens = sum(_lengths(case)) if "T" in case else B
    if case["op"] == "conv":  # input, output, state in and out, weights and bias
        return {"bytes": 2 * tokens * D * e + 6 * B * D * e + D * 20, "flops": 12 * tokens * D}
    N, G = case["state"], case["groups"]
    wide = 4 if case["gate"] else 3  # u, dt, y and the gate
    # one token of a state: decay, input and readout (7 operations, the exponential one of them)
    return {"bytes": tokens * (wide * D + 2 * G * N) * e + 8 * B * D * N + 4 * D * N + 8 * D, "flops": tokens * D * (7 * N + 24)}


# ---- inputs -----------------------------------------------------------------------------------
_TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(1_000_003 * int(seed) + 29)
    return g


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)


def _uniform(shape, g, lo, hi):
    return torch.rand(shape, generator=g, device=DEVICE) * (hi - lo) + lo


def prepare(case, seed):
    g = _generator(seed)
    return {"norm": _prepare_norm, "conv": _prepare_conv, "scan": _prepare_layer, "step": _prepare_layer}[case["op"]](case, g)


def _prepare_norm(case, g):
    n, d = case["rows"], case["width"]
    state = {"case": case, "x": _randn((n, d), g, _TYPE[case["x"]]), "weight": 1 + 0.1 * _randn((d,), g),
             "residual": None, "o": torch.empty((n, d), dtype=_TYPE[case["out"]], device=DEVICE), "scales": None}
    if case["residual"] != "none":
        state["residual"] = (4 * _randn((n, d), g)).to(_TYPE[case["residual"]])
    if case["out"] == "e4m3":
        groups = -(-d // case["group"]) if case["group"] else 1
        state["scales"] = torch.empty((n, groups), dtype=torch.float32, device=DEVICE)
    return state


def _slots(case, g):
    """A slot each of a pool with a few more, and the prompts' lengths (None: all of T)."""
    batch = case["batch"]
    pool = batch + 3
    slot = torch.randperm(pool, generator=g, device=DEVICE)[:batch].to(torch.int32)
    lens = None
    if case.get("ragged"):
        order = torch.randperm(batch, generator=g, device=DEVICE)
        lens = torch.tensor(_lengths(case), dtype=torch.int32, device=DEVICE)[order].contiguous()
    return pool, slot, lens


def _prepare_conv(case, g):
    B, T, D, dtype = case["batch"], case["T"], case["channels"], _TYPE[case["x"]]
    pool, slot, lens = _slots(case, g)
    # the layer's input projection gives the convolution's channels and the gate's side by side
    mixed = _randn((B, T, 2 * D), g, dtype)
    return {"case": case, "x": mixed[..., :D], "weight": 0.5 * _randn((D, 4), g), "bias": 0.1 * _randn((D,), g),
            "pool": _randn((pool, D, 3), g, dtype), "slot": slot, "lens": lens, "o": torch.zeros((B, T, D), dtype=dtype, device=DEVICE)}


def _prepare_layer(case, g):
    """Inputs of scan and step: [batch, T, ..] for the one, [batch, ..] for the other."""
    B, D, N, G, dtype = case["batch"], case["channels"], case["state"], case["groups"], _TYPE[case["x"]]
    at = (B, case["T"]) if case["op"] == "scan" else (B,)
    pool, slot, lens = _slots(case, g)
    rank = max(8, D // 16 // 8 * 8)
    mixed = _randn(at + (rank + 2 * G * N,), g, dtype)  # the projection that gives b and c beside dt's low-rank form
    step = torch.exp(_uniform((D,), g, math.log(0.001), math.log(0.1)))
    state = {"case": case, "u": _randn(at + (D,), g, dtype), "dt": (0.5 * _randn(at + (D,), g)).to(dtype),
             "a": -torch.arange(1, N + 1, device=DEVICE).float() * torch.exp(0.2 * _randn((D, N), g)),
             "b": mixed[..., rank:rank + G * N].unflatten(-1, (G, N)), "c": mixed[..., rank + G * N:].unflatten(-1, (G, N)),
             "z": _randn(at + (2 * D,), g, dtype)[..., D:] if case["gate"] else None,
             "skip": 1 + 0.1 * _randn((D,), g), "bias": step + torch.log(-torch.expm1(-step)),  # softplus(bias) = step
             "state": _randn((pool, D, N), g), "slot": slot, "lens": lens, "y": torch.zeros(at + (D,), dtype=dtype, device=DEVICE),
             "workspace": None}
    return state


# ---- one pass ---------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "conv": _own_conv, "scan": _own_scan, "step": _own_step}[op](state)
    return {"norm": _plain_norm, "conv": _plain_conv, "scan": _plain_scan, "step": _plain_step}[op](state)


def _norm_out(s):
    return {k: s[k] for k in ("o", "scales", "residual") if s[k] is not None}


def _own_norm(s):
    import linear_attention_decode_gdn_gb300 as gdn
    gdn.add_rms_norm(s["x"], s["o"], residual=s["residual"], weight=s["weight"], eps=EPS, scales=s["scales"], group=s["case"]["group"])
    return _norm_out(s)


def _own_conv(s):
    import linear_attention_decode_gdn_gb300 as gdn
    gdn.causal_conv(s["x"], s["weight"], s["pool"], s["slot"], s["o"], bias=s["bias"], seq_lens=s["lens"])
    return {"o": s["o"], "pool": s["pool"]}


def _own_scan(s):
    import linear_attention_decode_gdn_gb300 as gdn
    if s["workspace"] is None:  # scratch memory that a program allocates once
        size = gdn.ssm_workspace_bytes(*s["u"].shape, s["case"]["state"])
        s["workspace"] = torch.empty(max(16, size), dtype=torch.uint8, device=DEVICE)
    gdn.ssm_scan(s["u"], s["dt"], s["a"], s["b"], s["c"], s["state"], s["slot"], s["y"], s["workspace"], z=s["z"], skip=s["skip"],
                 dt_bias=s["bias"], seq_lens=s["lens"])
    return {"y": s["y"], "state": s["state"]}


def _own_step(s):
    import linear_attention_decode_gdn_gb300 as gdn
    gdn.ssm_step(s["u"], s["dt"], s["a"], s["b"], s["c"], s["state"], s["slot"], s["y"], z=s["z"], skip=s["skip"], dt_bias=s["bias"])
    return {"y": s["y"], "state": s["state"]}


def _plain_norm(s):
    x, d, group = s["x"].float(), s["case"]["width"], s["case"]["group"]
    if s["residual"] is not None:
        x = x + s["residual"].float()
        s["residual"].copy_(x)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["scales"] is None:
        s["o"].copy_(y)
        return _norm_out(s)
    wide = group or d
    rows = torch.nn.functional.pad(y, (0, -d % wide)).unflatten(-1, (-1, wide))
    s["scales"].copy_(rows.abs().amax(-1).clamp(min=LEAST) / TOP)
    s["o"].copy_((rows / s["scales"][..., None]).clamp(-TOP, TOP).flatten(-2)[:, :d])
    return _norm_out(s)


def _plain_conv(s):
    x, slot, T = s["x"], s["slot"].long(), s["x"].shape[1]
    joined = torch.cat([s["pool"][slot].transpose(1, 2), x], 1)  # the three inputs before, then the prompt
    wide = joined.float()
    o = s["bias"] + sum(wide[:, j:j + T] * s["weight"][:, j] for j in range(4))
    o = o * torch.sigmoid(o)
    lens = s["lens"].long() if s["lens"] is not None else torch.full_like(slot, T)
    live = torch.arange(T, device=DEVICE) < lens[:, None]
    s["o"].copy_(torch.where(live[..., None], o, s["o"].float()))
    last = (lens[:, None] + torch.arange(3, device=DEVICE))[..., None].expand(-1, -1, x.shape[2])
    s["pool"][slot] = joined.gather(1, last).transpose(1, 2)
    return {"o": s["o"], "pool": s["pool"]}


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _per_channel(x, D):
    """[.., groups, N] to [.., D, N]: each group's row for all its channels."""
    return x.float().repeat_interleave(D // x.shape[-2], dim=-2)


def _readout(s, states, y):
    """y + skip u, gated, from the states' readout."""
    y = y + s["skip"] * s["u"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y


def _plain_step(s):
    slot, D = s["slot"].long(), s["case"]["channels"]
    dt = _softplus(s["dt"].float() + s["bias"])
    h = s["state"][slot] * torch.exp(dt[..., None] * s["a"]) + (dt * s["u"].float())[..., None] * _per_channel(s["b"], D)
    s["state"][slot] = h
    s["y"].copy_(_readout(s, h, (h * _per_channel(s["c"], D)).sum(-1)))
    return {"y": s["y"], "state": s["state"]}


def _plain_scan(s):
    slot, D, T = s["slot"].long(), s["case"]["channels"], s["case"]["T"]
    dt = _softplus(s["dt"].float() + s["bias"])
    live = None
    if s["lens"] is not None:
        live = torch.arange(T, device=DEVICE) < s["lens"][:, None]
        dt = dt * live[..., None]  # a position past the prompt leaves the state as it is
    decay = torch.exp(dt[..., None] * s["a"])  # [batch, T, D, N]
    h = (dt * s["u"].float())[..., None] * _per_channel(s["b"], D)
    h[:, 0] += decay[:, 0] * s["state"][slot]
    reach = 1
    while reach < T:  # h of a position holds its last `reach` inputs, decay their product: both double
        h[:, reach:] += decay[:, reach:] * h[:, :-reach]
        decay[:, reach:] = decay[:, reach:] * decay[:, :-reach]
        reach *= 2
    s["state"][slot] = h[:, -1]
    y = _readout(s, h, (h * _per_channel(s["c"], D)).sum(-1))
    s["y"].copy_(y if live is None else torch.where(live[..., None], y, s["y"].float()))
    return {"y": s["y"], "state": s["state"]}


# ---- the definition, in 64 bits -----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan, "step": _exact_scan}[case["op"]](s)


def _exact_norm(s):
    total = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    power = torch.einsum("nd,nd->n", total, total) / total.shape[1]
    y = total / torch.sqrt(power + EPS)[:, None] * s["weight"].double()
    out = {"o": y}
    if s["residual"] is not None:
        out["residual"] = total
    if s["scales"] is not None:
        wide = s["case"]["group"] or y.shape[1]
        pieces = y.split(wide, 1)
        out["scales"] = torch.stack([p.abs().max(1).values.clamp(min=LEAST) / TOP for p in pieces], 1)
        out["o"] = torch.cat([p / out["scales"][:, i, None] for i, p in enumerate(pieces)], 1)
    return out


def _exact_conv(s):
    o, pool = s["o"].double(), s["pool"].double()
    w, bias = s["weight"].double(), s["bias"].double()
    lens = s["lens"].tolist() if s["lens"] is not None else [s["x"].shape[1]] * s["x"].shape[0]
    for i, (row, n) in enumerate(zip(s["slot"].tolist(), lens)):
        line = torch.cat([pool[row].T, s["x"][i, :n].double()])
        taps = torch.nn.functional.conv1d(line.T[None], w[:, None], bias, groups=w.shape[0])[0].T
        o[i, :n] = taps / (1 + torch.exp(-taps))
        pool[row] = line[n:].T
    return {"o": o, "pool": pool}


def _exact_scan(s):
    single = s["case"]["op"] == "step"
    of = lambda name: s[name].double()[:, None] if single else s[name].double()  # noqa: E731
    D, G = s["case"]["channels"], s["case"]["groups"]
    rows, lens = s["slot"].long(), s["lens"]
    u, b, c = of("u"), of("b"), of("c")
    dt = torch.nn.functional.softplus(of("dt") + s["bias"].double(), threshold=200)
    a, h = s["a"].double(), s["state"].double()[rows]
    y = of("y").clone()
    for t in range(u.shape[1]):
        take = dt[:, t, :, None]
        new = torch.exp(take * a) * h
        new += ((take[..., 0] * u[:, t]).unflatten(1, (G, D // G))[..., None] * b[:, t, :, None]).flatten(1, 2)
        row = (new.unflatten(1, (G, D // G)) * c[:, t, :, None]).sum(-1).flatten(1) + s["skip"].double() * u[:, t]
        if s["z"] is not None:
            z = of("z")[:, t] if single else s["z"][:, t].double()
            row = row * z / (1 + torch.exp(-z))
        if lens is None:
            h, y[:, t] = new, row
        else:
            live = (t < lens)[:, None]
            h, y[:, t] = torch.where(live[..., None], new, h), torch.where(live, row, y[:, t])
    state = s["state"].double()
    state[rows] = h
    return {"y": y[:, 0] if single else y, "state": state}
