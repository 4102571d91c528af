"""The paged-cache operators in their plain form, and the cases they are measured on.

Four operators that run one decode step of an attention layer next to the recurrent ones:

* ``plan``   block tables and slot maps from the requests' lengths,
* ``append`` the new tokens' keys and values (or latent rows) written into their pages,
* ``attn``   grouped-query attention of the newest 1..T tokens of each request over its pages,
* ``latent`` the same over one shared latent row a token (the value is the row's first part).

``run`` computes an operator with elementary torch operations where ``own`` is false, and with the
library's calls where it is true.
"""
import math

import torch

own = False

DEVICE = "cuda"
LATENT, TAIL = 512, 64  # a latent row: the shared latent, then the positional part of the key


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a full batch: nearly every token lands in a page that is already held
        {"name": "plan_decode", "op": "plan", "batch": 256, "ctx": 8191, "new": 1, "page": 64},
        # prompts admitted together: ragged, some requests idle, many pages handed out
        {"name": "plan_prompts", "op": "plan", "batch": 512, "ctx": 1000, "new": 511, "page": 16},
        # the write of one decode step
        {"name": "append_decode", "op": "append", "tokens": 128, "heads_kv": 8, "dk": 128, "page": 64, "latent": False, "fp32": False},
        # the write of long prompts: keys and values, a few padded rows
        {"name": "append_prompts", "op": "append", "tokens": 32749, "heads_kv": 8, "dk": 128, "page": 16, "latent": False, "fp32": False},
        # latent rows of prompts, from fp32 projections
        {"name": "append_latent", "op": "append", "tokens": 16381, "heads_kv": 1, "dk": LATENT + TAIL, "page": 64, "latent": True, "fp32": True},
        # one user, a short context: latency
        {"name": "attn_single", "op": "attn", "batch": 1, "T": 1, "heads": 16, "heads_kv": 2, "dk": 256, "ctx": 1021, "ragged": False, "page": 64, "window": 0},
        # a full batch with contexts of every length
        {"name": "attn_batch", "op": "attn", "batch": 128, "T": 1, "heads": 32, "heads_kv": 8, "dk": 128, "ctx": 8190, "ragged": True, "page": 64, "window": 0},
        # one user with a very long context: the work has to be split along it
        {"name": "attn_long", "op": "attn", "batch": 1, "T": 1, "heads": 32, "heads_kv": 8, "dk": 128, "ctx": 131071, "ragged": False, "page": 128, "window": 0},
        # speculative verification of four positions, sliding window, small pages
        {"name": "attn_verify", "op": "attn", "batch": 32, "T": 4, "heads": 16, "heads_kv": 4, "dk": 64, "ctx": 6143, "ragged": True, "page": 16, "window": 4096},
        # two users on latent rows: latency
        {"name": "latent_small", "op": "latent", "batch": 2, "T": 1, "heads": 16, "ctx": 701, "ragged": False, "page": 64, "window": 0},
        # a full batch on latent rows
        {"name": "latent_batch", "op": "latent", "batch": 128, "T": 1, "heads": 32, "ctx": 8190, "ragged": True, "page": 64, "window": 0},
        # four long contexts and many heads: as much arithmetic as traffic
        {"name": "latent_long", "op": "latent", "batch": 4, "T": 1, "heads": 128, "ctx": 65535, "ragged": False, "page": 32, "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "latent", "latent"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        new = rng.choice([1, _log(rng, 2, 511)])
        return {"op": op, "batch": _log(rng, 1, 512), "ctx": _log(rng, 1, 8191), "new": new, "page": page}
    if op == "append":
        latent = rng.random() < 0.4
        return {"op": op, "tokens": _log(rng, 1, 32749 if not latent else 16381), "heads_kv": 1 if latent else rng.choice([1, 2, 4, 8]),
                "dk": LATENT + TAIL if latent else rng.choice([64, 128]), "page": page, "latent": latent, "fp32": rng.random() < 0.4}
    T = rng.choice([1, 1, 2, 3, 4])
    window = rng.choice([0, 0, 0, _log(rng, 1, 8191)])
    ragged = rng.random() < 0.6
    if op == "latent":
        heads = rng.choice([8, 16, 20, 32, 64, 128])
        while True:
            batch, ctx = _log(rng, 1, 128), _log(rng, 1, 65535)
            if batch * ctx * max(1, heads * T // 32) <= 128 * 8190:
                break
        return {"op": op, "batch": batch, "T": T, "heads": heads, "ctx": ctx, "ragged": ragged, "page": page, "window": window}
    dk = rng.choice([64, 128, 128, 256])
    heads_kv = rng.choice([1, 2, 4, 8])
    heads = heads_kv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    while True:
        batch, ctx = _log(rng, 1, 128), _log(rng, 1, 131071)
        if batch * ctx * heads_kv * dk * max(1, heads // heads_kv * T // 16) <= 64 * 8190 * 8 * 128:
            break
    return {"op": op, "batch": batch, "T": T, "heads": heads, "heads_kv": heads_kv, "dk": dk, "ctx": ctx, "ragged": ragged, "page": page, "window": window}


def _lengths(case):
    """The cached lengths of the requests, before a permutation: the same for every seed."""
    batch, ctx = case["batch"], case["ctx"]
    if case.get("ragged", True):  # evenly from ctx down to about ctx / batch
        return [ctx - ctx * i // batch for i in range(batch)]
    return [max(0, ctx - i % 7) for i in range(batch)]


def _news(case):
    if case["new"] == 1:
        return [1] * case["batch"]
    return [case["new"] * ((5 * i) % 8) // 7 for i in range(case["batch"])]


def _shape(case):
    """(query heads, kv heads, key size, value size) of an attention case."""
    if case["op"] == "latent":
        return case["heads"], 1, LATENT + TAIL, LATENT
    return case["heads"], case["heads_kv"], case["dk"], case["dk"]


def work(case):
    if case["op"] == "plan":
        new, length = sum(_news(case)), _lengths(case)
        last = [-(-(c + n) // case["page"]) for c, n in zip(length, _news(case))]
        extra = sum(n - -(-c // case["page"]) for c, n in zip(length, last))
        # lengths and page counts in and out, offsets, one slot a token, the pages handed out
        return {"bytes": 4 * 6 * case["batch"] + 8 * new + 8 * extra + 4 * new / case["page"], "flops": 0}
    if case["op"] == "append":
        width = case["heads_kv"] * case["dk"] * (1 if case["latent"] else 2)
        return {"bytes": case["tokens"] * (width * ((4 if case["fp32"] else 2) + 2) + 8), "flops": 0}
    heads, heads_kv, dk, dv = _shape(case)
    T, window = case["T"], case["window"]
    read = [min(n, window + T - 1) if window else n for n in _lengths(case)]
    row = heads_kv * (dk + dv) if case["op"] == "attn" else dk
    pairs = sum(sum(max(0, min(n - T + t + 1, window or n)) for t in range(T)) for n in _lengths(case))
    rows = case["batch"] * T * heads
    return {"bytes": sum(read) * row * 2 + rows * (dk + dv) * 2 + rows * 4 + sum(-(-n // case["page"]) for n in read) * 4 + 4 * case["batch"],
            "flops": 2 * pairs * heads * (dk + dv)}


# ---- inputs -----------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(1_000_003 * int(seed) + 17)
    return g


def _randn(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _pages(lengths, page, g, spare=3):
    """A block table over shuffled pages, -1 past each request's own, and the pages that are left."""
    count = (lengths + page - 1) // page
    need, widest = int(count.sum()), int(count.max())
    total = need + spare
    perm = torch.randperm(total, generator=g, device=DEVICE).to(torch.int32)
    start = torch.cumsum(count, 0) - count
    column = torch.arange(max(1, widest), device=DEVICE)
    held = column[None, :] < count[:, None]
    table = torch.where(held, perm[(start[:, None] + column).clamp(max=total - 1)], -1).to(torch.int32)
    return table, perm[need:].contiguous(), total


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, g)
    if case["op"] == "append":
        return _prepare_append(case, g)
    heads, heads_kv, dk, dv = _shape(case)
    batch, T, page = case["batch"], case["T"], case["page"]
    length = _int(_lengths(case))[torch.randperm(batch, generator=g, device=DEVICE)]
    table, _, total = _pages(length, page, g)
    state = {"case": case, "q": _randn((batch, T, heads, dk), g), "table": table, "length": length,
             "k": _randn((total, page, heads_kv, dk), g),
             "o": torch.empty((batch, T, heads, dv), dtype=torch.bfloat16, device=DEVICE),
             "lse": torch.empty((batch, T, heads), dtype=torch.float32, device=DEVICE),
             "scale": dk ** -0.5, "window": case["window"], "workspace": None}
    if case["op"] == "attn":
        state["v"] = _randn((total, page, heads_kv, dv), g)
    return state


def _prepare_plan(case, g):
    order = torch.randperm(case["batch"], generator=g, device=DEVICE)
    cached, new = _int(_lengths(case))[order], _int(_news(case))[order]
    page = case["page"]
    table, _, used = _pages(cached, page, g, spare=0)
    widest = -(-(case["ctx"] + max(_news(case))) // page)
    room = torch.full((case["batch"], widest), -1, dtype=torch.int32, device=DEVICE)
    room[:, :table.shape[1]] = table[:, :widest]
    held = (cached + page - 1) // page
    wanted = int(((cached + new + page - 1) // page - held).sum())
    total = used + wanted + 5
    free = used + torch.randperm(total - used, generator=g, device=DEVICE).to(torch.int32)
    tokens = max(1, sum(_news(case)))
    empty = lambda n, t=torch.int32: torch.empty(n, dtype=t, device=DEVICE)  # noqa: E731
    return {"case": case, "cached": cached, "new": new, "held": held, "table": room, "free": free,
            "free_count": _int([total - used]), "num_pages": total, "page": page,
            "length": empty(case["batch"]), "offsets": empty(case["batch"] + 1), "slots": empty(tokens, torch.int64),
            "held_out": empty(case["batch"]), "free_out": empty(1)}


def _prepare_append(case, g):
    n, page = case["tokens"], case["page"]
    pages = -(-n // page) + 2
    slots = torch.randperm(pages * page, generator=g, device=DEVICE)[:n] if n % 2 else torch.arange(n, device=DEVICE) + page
    slots = slots.to(torch.int64).contiguous()
    if n > 64:
        slots[torch.randint(0, n, (n // 64,), generator=g, device=DEVICE)] = -1  # padded rows
    dtype = torch.float32 if case["fp32"] else torch.bfloat16
    state = {"case": case, "slots": slots, "pool_k": _randn((pages, page, case["heads_kv"], case["dk"]), g)}
    if case["latent"]:
        state["k"], state["v"] = _randn((n, 1, LATENT), g, dtype), _randn((n, 1, TAIL), g, dtype)
    else:
        # the two are slices of one projection's rows
        mixed = _randn((n, 2 * case["heads_kv"], case["dk"]), g, dtype)
        state["k"], state["v"] = mixed[:, :case["heads_kv"]], mixed[:, case["heads_kv"]:]
        state["pool_v"] = _randn((pages, page, case["heads_kv"], case["dk"]), g)
    return state


# ---- one pass ---------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "attn": _own_attend, "latent": _own_attend}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attend, "latent": _plain_attend}[op](state)


def _own_plan(s):
    import linear_attention_decode_gdn_gb300 as gdn
    gdn.kv_plan(s["cached"], s["new"], s["held"], s["table"], s["free"], s["free_count"], kv_len=s["length"], cu_new=s["offsets"],
                slot_map=s["slots"], held_out=s["held_out"], free_count_out=s["free_out"], page_size=s["page"], num_pages=s["num_pages"])
    return {"length": s["length"], "offsets": s["offsets"], "slots": s["slots"], "table": s["table"], "held": s["held_out"], "free": s["free_out"]}


def _own_append(s):
    import linear_attention_decode_gdn_gb300 as gdn
    latent = s["case"]["latent"]
    kv = gdn.make_paged_kv(s["pool_k"], dv=LATENT) if latent else gdn.make_paged_kv(s["pool_k"], s["pool_v"])
    gdn.kv_append(kv, s["k"], s["v"], s["slots"])
    return {"k": s["pool_k"]} if latent else {"k": s["pool_k"], "v": s["pool_v"]}


def _own_attend(s):
    import linear_attention_decode_gdn_gb300 as gdn
    latent = s["case"]["op"] == "latent"
    kv = gdn.make_paged_kv(s["k"], dv=LATENT) if latent else gdn.make_paged_kv(s["k"], s["v"])
    if s["workspace"] is None:  # scratch memory that a program allocates once
        size = gdn.attn_workspace_bytes(kv, *s["q"].shape[:3])
        s["workspace"] = torch.empty(max(16, size), dtype=torch.uint8, device=DEVICE)
    call = gdn.latent_decode if latent else gdn.attn_decode
    call(kv, s["q"], s["table"], s["length"], s["o"], s["workspace"], lse=s["lse"], scale=s["scale"], window=s["window"])
    return {"o": s["o"], "lse": s["lse"]}


def _plain_plan(s):
    cached, new, held, page = s["cached"].long(), s["new"].long(), s["held"].long(), s["page"]
    avail = s["free_count"].long()
    want = ((cached + new + page - 1) // page - held).clamp(min=0)
    upto = torch.cumsum(want, 0)
    fits = (upto <= avail) | (want == 0)
    rank = upto - want
    column = torch.arange(s["table"].shape[1], device=DEVICE)
    fresh = (column >= held[:, None]) & (column < (held + want)[:, None]) & fits[:, None]
    at = (avail - 1 - (rank - held)[:, None] - column).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    offsets = torch.cat([torch.zeros_like(avail), torch.cumsum(new, 0)])
    token = torch.arange(s["slots"].numel(), device=DEVICE)
    b = torch.searchsorted(offsets[1:], token, right=True).clamp(max=cached.numel() - 1)
    position = cached[b] + token - offsets[b]
    slot = table[b, (position // page).clamp(max=table.shape[1] - 1)].long() * page + position % page
    slot = torch.where((token < offsets[-1]) & fits[b], slot, -1)
    return {"length": torch.where(fits, cached + new, cached).int(), "offsets": offsets.int(), "slots": slot, "table": table,
            "held": torch.where(fits, held + want, held).int(), "free": (avail - torch.where(fits, want, 0).sum()).int()}


def _plain_append(s):
    live = s["slots"] >= 0
    to = s["slots"][live]
    if s["case"]["latent"]:
        rows = torch.cat([s["k"], s["v"]], dim=-1)
        s["pool_k"].view(-1, *s["pool_k"].shape[2:])[to] = rows[live].to(torch.bfloat16)
        return {"k": s["pool_k"]}
    s["pool_k"].view(-1, *s["pool_k"].shape[2:])[to] = s["k"][live].to(torch.bfloat16)
    s["pool_v"].view(-1, *s["pool_v"].shape[2:])[to] = s["v"][live].to(torch.bfloat16)
    return {"k": s["pool_k"], "v": s["pool_v"]}


def _plain_attend(s):
    heads, heads_kv, dk, dv = _shape(s["case"])
    q, length = s["q"], s["length"].long()
    batch, T = q.shape[:2]
    group = heads // heads_kv
    table = s["table"].long().clamp(min=0)
    k = s["k"][table].float().flatten(1, 2).transpose(1, 2)  # [batch, heads_kv, positions, dk]
    v = s["v"][table].float().flatten(1, 2).transpose(1, 2) if "v" in s else k[..., :dv]
    position = torch.arange(k.shape[2], device=DEVICE)
    last = (length[:, None] - T + torch.arange(T, device=DEVICE))[:, :, None]  # each query's own position
    seen = position <= last
    if s["window"]:
        seen = seen & (position > last - s["window"])
    qg = q.float().view(batch, T, heads_kv, group, dk).permute(0, 2, 1, 3, 4).reshape(batch, heads_kv, T * group, dk)
    score = torch.matmul(qg, k.transpose(2, 3)) * s["scale"]
    seen = seen[:, None, :, None, :].expand(batch, 1, T, group, -1).reshape(batch, 1, T * group, -1)
    score = score.masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top.clamp(min=-3e38))
    total = weight.sum(-1, keepdim=True)
    o = torch.matmul(weight, v) / total.clamp(min=1e-38)
    lse = (top + torch.log(total))[..., 0]
    lse = torch.where(total[..., 0] > 0, lse, float("-inf"))
    o = o.view(batch, heads_kv, T, group, dv).permute(0, 2, 1, 3, 4).reshape(batch, T, heads, dv)
    lse = lse.view(batch, heads_kv, T, group).permute(0, 2, 1, 3).reshape(batch, T, heads)
    return {"o": o.to(torch.bfloat16), "lse": lse}


# ---- the definition, in 64 bits -----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] == "append":
        return _exact_append(s)
    heads, heads_kv, dk, dv = _shape(case)
    batch, T, group = case["batch"], case["T"], heads // heads_kv
    o = torch.zeros((batch, T, heads, dv), dtype=torch.float64, device=DEVICE)
    lse = torch.full((batch, T, heads), float("-inf"), dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(s["length"].tolist()):
        if n == 0:
            continue
        own_pages = s["table"][b, :-(-n // case["page"])].long()
        k = s["k"][own_pages].flatten(0, 1)[:n].double()
        v = s["v"][own_pages].flatten(0, 1)[:n].double() if case["op"] == "attn" else k[..., :dv]
        for t in range(T):
            end = n - T + t + 1
            begin = max(0, end - case["window"]) if case["window"] else 0
            if end <= begin:
                continue
            for j in range(heads_kv):
                rows = slice(j * group, (j + 1) * group)
                x = s["q"][b, t, rows].double() @ k[begin:end, j].T * s["scale"]
                lse[b, t, rows] = torch.logsumexp(x, -1)
                o[b, t, rows] = torch.softmax(x, -1) @ v[begin:end, j]
    return {"o": o, "lse": lse}


def _exact_append(s):
    to = s["slots"].tolist()
    live = [i for i, x in enumerate(to) if x >= 0]
    index = torch.tensor([to[i] for i in live], dtype=torch.int64, device=DEVICE)
    source = torch.tensor(live, dtype=torch.int64, device=DEVICE)
    pools = {"k": s["pool_k"].double().flatten(0, 1)}
    if s["case"]["latent"]:
        pools["k"][index, :, :LATENT] = s["k"].double()[source]
        pools["k"][index, :, LATENT:] = s["v"].double()[source]
        return {"k": pools["k"].view(s["pool_k"].shape)}
    pools["v"] = s["pool_v"].double().flatten(0, 1)
    pools["k"].index_copy_(0, index, s["k"].double()[source])
    pools["v"].index_copy_(0, index, s["v"].double()[source])
    return {name: pool.view(s["pool_k"].shape) for name, pool in pools.items()}
