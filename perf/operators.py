"""Sequence operators: what is measured.

Two operators over token sequences, each in its three forms:

- window attention: query at position p sees the keys p - window < j <= p and
  the first `sinks` keys; grouped heads; prompts (whole, or a chunk of new
  tokens behind a cache), single tokens over a cache, and training.
- linear attention with a decay for each head:
  S_t = exp(log_decay) S_(t-1) + k_t v_t^T, o_t = scale q_t S_t; prompts,
  single tokens (the state updated in place) and training.

`run` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with `own`, through the package.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One short request with a small model's heads: the latency of a prompt call.
        {"name": "window prompt short", "op": "window", "form": "prompt", "dtype": "fp16", "B": 1, "Lq": 200, "Lk": 200,
         "Hq": 8, "Hkv": 2, "D": 64, "window": 64, "sinks": 4, "page": 0, "ragged": False},
        # A long document read in one call: the largest prompt.
        {"name": "window prompt long", "op": "window", "form": "prompt", "dtype": "bf16", "B": 1, "Lq": 16384, "Lk": 16384,
         "Hq": 32, "Hkv": 8, "D": 128, "window": 2048, "sinks": 4, "page": 0, "ragged": False},
        # Several prompts of different lengths, each continued by a chunk of new tokens over a paged cache.
        {"name": "window prompt chunk paged", "op": "window", "form": "prompt", "dtype": "fp16", "B": 6, "Lq": 509, "Lk": 4001,
         "Hq": 16, "Hkv": 4, "D": 80, "window": 1000, "sinks": 17, "page": 16, "ragged": True},
        # One user's next token over a long cache: latency again, one row for each head.
        {"name": "window step one", "op": "window", "form": "step", "dtype": "bf16", "B": 1, "Lq": 1, "Lk": 8192,
         "Hq": 32, "Hkv": 8, "D": 128, "window": 4096, "sinks": 4, "page": 0, "ragged": False},
        # The next token of a full serving batch over pages.
        {"name": "window step batch paged", "op": "window", "form": "step", "dtype": "bf16", "B": 64, "Lq": 1, "Lk": 8192,
         "Hq": 32, "Hkv": 8, "D": 128, "window": 2048, "sinks": 16, "page": 64, "ragged": True},
        # A training step of a small model on odd lengths.
        {"name": "window train odd", "op": "window", "form": "train", "dtype": "fp16", "B": 2, "Lq": 777, "Lk": 777,
         "Hq": 6, "Hkv": 3, "D": 64, "window": 131, "sinks": 5, "page": 0, "ragged": False},
        # A training step on long sequences.
        {"name": "window train long", "op": "window", "form": "train", "dtype": "bf16", "B": 1, "Lq": 8192, "Lk": 8192,
         "Hq": 16, "Hkv": 4, "D": 128, "window": 1024, "sinks": 4, "page": 0, "ragged": False},
        # A short prompt with few heads.
        {"name": "linear prompt short", "op": "linear", "form": "prompt", "dtype": "fp16", "B": 1, "L": 300,
         "H": 4, "Dk": 64, "Dv": 64, "ragged": False},
        # A long document with a state from before: few sequences, a long axis.
        {"name": "linear prompt long", "op": "linear", "form": "prompt", "dtype": "bf16", "B": 1, "L": 32768,
         "H": 16, "Dk": 128, "Dv": 128, "ragged": False},
        # One user's next token: latency.
        {"name": "linear step one", "op": "linear", "form": "step", "dtype": "bf16", "B": 1, "L": 1,
         "H": 16, "Dk": 128, "Dv": 128, "ragged": False},
        # The next token of a full serving batch.
        {"name": "linear step batch", "op": "linear", "form": "step", "dtype": "bf16", "B": 64, "L": 1,
         "H": 32, "Dk": 128, "Dv": 128, "ragged": False},
        # A training step on long sequences.
        {"name": "linear train long", "op": "linear", "form": "train", "dtype": "bf16", "B": 2, "L": 8192,
         "H": 16, "Dk": 128, "Dv": 128, "ragged": False},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    form = rng.choice(("prompt", "step", "train"))
    dtype = rng.choice(("bf16", "fp16"))
    if rng.random() < 0.55:
        Hkv, group, D = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 80, 96, 128))
        window, sinks = _spread(rng, 16, 4096), rng.choice((0, 1, 4, 7, 16, 33, 64))
        case = {"op": "window", "form": form, "dtype": dtype, "B": 1, "Lq": 1, "Lk": 1, "Hq": Hkv * group, "Hkv": Hkv, "D": D,
                "window": window, "sinks": sinks, "page": 0, "ragged": rng.random() < 0.5}
        if form == "step":
            case.update(B=_spread(rng, 1, 64), Lk=_spread(rng, 64, 8192), page=rng.choice((0, 16, 64)))
        elif form == "train":
            L = _spread(rng, 65, 8192)
            case.update(B=rng.choice((1, 2, 3)), Lq=L, Lk=L)
        else:
            L = _spread(rng, 65, 16384)
            case.update(B=rng.choice((1, 2, 4)), Lq=L, Lk=L, page=rng.choice((0, 0, 16, 64)))
            if rng.random() < 0.4:
                case["Lq"] = _spread(rng, 17, L)
        lk = "Lk"
    else:
        case = {"op": "linear", "form": form, "dtype": dtype, "B": rng.choice((1, 2, 3)), "L": 1, "H": _spread(rng, 1, 32),
                "Dk": rng.choice((64, 96, 128)), "Dv": rng.choice((64, 80, 128)), "ragged": form != "step" and rng.random() < 0.4}
        if form == "step":
            case["B"] = _spread(rng, 1, 64)
        else:
            case["L"] = _spread(rng, 65, 32768 if form == "prompt" else 8192)
        lk = "L"
    most = [c for c in listed() if c["op"] == case["op"] and c["form"] == form]
    while any(work(case)[m] > max(work(c)[m] for c in most) for m in ("bytes", "flops")):
        if case[lk] > 256:
            case[lk] = case[lk] * 3 // 4
            if case["op"] == "window":
                case["Lq"] = case["Lk"] if form == "train" else min(case["Lq"], case["Lk"])
        elif case["B"] > 1:
            case["B"] -= 1
        else:
            break
    return case


def _lengths(case, most):
    """Tokens of each sequence: the case alone decides."""
    B = case["B"]
    if not case["ragged"]:
        return [most] * B
    return [max(1, most - (most * 5 * ((3 * b + 1) % B)) // (7 * B) - b % 2) for b in range(B)]


def _visible(p, window, sinks):
    """Number of keys that the query at position p sees."""
    near = min(window, p + 1)
    return near + min(sinks, p + 1 - near)


def work(case):
    e = 2
    if case["op"] == "window":
        nk = _lengths(case, case["Lk"])
        nq = [min(case["Lq"], n) for n in nk]
        pairs = sum(_visible(n - m + i, case["window"], case["sinks"]) for n, m in zip(nk, nq) for i in range(m))
        # The keys that some query sees.
        keys = sum(min(n, case["window"] + m - 1 + min(case["sinks"], max(0, n - case["window"] - m + 1))) for n, m in zip(nk, nq))
        q, kv = sum(nq) * case["Hq"] * case["D"] * e, keys * case["Hkv"] * case["D"] * e
        flops = 4 * case["D"] * case["Hq"] * pairs
        if case["form"] == "train":  # forward and backward: q, k, v, dout in; out, dq, dk, dv out
            return {"bytes": 4 * q + 4 * kv, "flops": 3.5 * flops}
        return {"bytes": 2 * q + 2 * kv, "flops": flops}
    n, H, Dk, Dv = sum(_lengths(case, case["L"])), case["H"], case["Dk"], case["Dv"]
    tokens, state = n * H * (2 * Dk + 2 * Dv) * e, case["B"] * H * Dk * Dv * 4
    flops = 4 * n * H * Dk * Dv
    if case["form"] == "train":  # q, k, v, dout in; out, dq, dk, dv out
        return {"bytes": n * H * (4 * Dk + 4 * Dv) * e, "flops": 3 * flops}
    return {"bytes": tokens + 2 * state, "flops": flops}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    t = TYPES[case["dtype"]]

    def normal(*shape, dtype=t, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s, B = {"case": dict(case)}, case["B"]
    if case["op"] == "window":
        Hq, Hkv, D, Lq, Lk = case["Hq"], case["Hkv"], case["D"], case["Lq"], case["Lk"]
        s["scale"] = D ** -0.5
        nk = _lengths(case, Lk)
        s["q_lens"], s["kv_lens"], s["pages"] = None, None, None
        if case["ragged"]:
            s["q_lens"], s["kv_lens"] = ints([min(Lq, n) for n in nk]), ints(nk)
        if case["page"]:  # a cache in pages, handed out in a mixed order
            size = case["page"]
            per = -(-Lk // size)
            s["k"], s["v"] = normal(B * per, size, Hkv, D), normal(B * per, size, Hkv, D)
            s["pages"] = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).reshape(B, per)
            s["q"] = normal(B, Lq, Hq, D, std=1.5)
        elif case["form"] == "step" or Lq != Lk:  # a cache of whole sequences
            s["k"], s["v"] = normal(B, Lk, Hkv, D), normal(B, Lk, Hkv, D)
            s["q"] = normal(B, Lq, Hq, D, std=1.5)
        else:  # the three parts of one projection
            x = normal(B, Lk, (Hq + 2 * Hkv) * D)
            x[..., :Hq * D] *= 1.5
            s["q"], s["k"], s["v"] = (y.unflatten(2, (-1, D)) for y in x.split([Hq * D, Hkv * D, Hkv * D], 2))
        if case["form"] == "train":
            s["dout"] = normal(B, Lq, Hq, D)
        return s
    L, H, Dk, Dv = case["L"], case["H"], case["Dk"], case["Dv"]
    s["scale"] = Dk ** -0.5
    # Half-lives from one token to some hundreds, spread over the heads.
    s["log_decay"] = -torch.exp2(-8.0 * (torch.arange(H, device="cuda", dtype=torch.float32) + 1) / H)
    if case["form"] == "step":
        s["q"], s["k"], s["v"] = normal(B, H, Dk), normal(B, H, Dk), normal(B, H, Dv)
    else:  # the three parts of one projection
        x = normal(B, L, H * (2 * Dk + Dv))
        s["q"], s["k"], s["v"] = (y.unflatten(2, (H, -1)) for y in x.split([H * Dk, H * Dk, H * Dv], 2))
    s["lens"] = ints(_lengths(case, L)) if case["ragged"] else None
    if case["form"] == "train":
        s["dout"] = normal(B, L, H, Dv)
    else:
        s["state"] = normal(B, H, Dk, Dv, dtype=torch.float32, std=2.0)
    return s


def run(state):
    if own:
        return _run_own(state)
    if state["case"]["op"] == "window":
        return _plain_window(state)
    return _plain_linear(state)


def _run_own(s):
    import memory_efficient_im2win_amd as m
    case, form = s["case"], s["case"]["form"]
    if case["op"] == "window":
        args = dict(window=case["window"], sinks=case["sinks"], scale=s["scale"], q_lens=s["q_lens"], kv_lens=s["kv_lens"])
        if form != "train":
            return m.window_attention(s["q"], s["k"], s["v"], page_table=s["pages"], **args)
        out, lse = m.window_attention(s["q"], s["k"], s["v"], return_lse=True, **args)
        return (out,) + tuple(m.window_attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **args))
    if form == "step":
        return m.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"]), s["state"]
    if form == "prompt":
        return m.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], scale=s["scale"], lens=s["lens"])
    out, _ = m.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], lens=s["lens"])
    dq, dk, dv, _ = m.linear_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], lens=s["lens"])
    return out, dq, dk, dv


# ---- plain forms -------------------------------------------------------------
def _window_lengths(s):
    case, dev = s["case"], s["q"].device
    if s["kv_lens"] is not None:
        return s["q_lens"].long(), s["kv_lens"].long()
    return torch.full((case["B"],), case["Lq"], device=dev), torch.full((case["B"],), case["Lk"], device=dev)


def _plain_window(s):
    """Queries in blocks of C; for each block the run of keys that its windows
    cover, gathered, and the sinks beside them."""
    case, t = s["case"], s["q"].dtype
    B, Lq, Hq, D = s["q"].shape
    Hkv, W, sinks = case["Hkv"], case["window"], case["sinks"]
    G, dev = Hq // Hkv, s["q"].device
    C = min(Lq, max(64, W))
    N = -(-Lq // C)
    nq, nk = _window_lengths(s)
    row = torch.arange(N * C, device=dev).view(1, N, C)
    pos = (nk - nq).view(B, 1, 1) + row
    pos = torch.where(row < nq.view(B, 1, 1), pos, -1)  # (B, N, C); nothing is visible from -1
    first = (nk - nq).view(B, 1) + torch.arange(N, device=dev) * C - W + 1
    near = first.unsqueeze(2) + torch.arange(W + C - 1, device=dev)  # (B, N, W + C - 1)
    far = torch.arange(sinks, device=dev).expand(B, N, sinks)
    key = torch.cat([far, near], 2)  # (B, N, M)
    p, j = pos.unsqueeze(3), key.unsqueeze(2)
    in_window = (j >= 0) & (j <= p) & (j > p - W)
    in_sinks = (j <= p - W) & (j < nk.view(B, 1, 1, 1))
    is_far = torch.arange(key.shape[2], device=dev) < sinks
    seen = torch.where(is_far, in_sinks, in_window).unsqueeze(2).unsqueeze(3)  # (B, N, 1, 1, C, M)
    at = key.clamp(0, case["Lk"] - 1)
    batch = torch.arange(B, device=dev).view(B, 1, 1)
    if s["pages"] is not None:
        size = case["page"]
        page = s["pages"].long()[batch, at // size]
        k, v = s["k"][page, at % size], s["v"][page, at % size]
    else:
        k, v = s["k"][batch, at], s["v"][batch, at]

    def blocks(x):  # (B, Lq, Hq, D) to (B, N, Hkv, G * C, D)
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, N * C - Lq))
        return x.view(B, N, C, Hkv, G, D).permute(0, 1, 3, 4, 2, 5).reshape(B, N, Hkv, G * C, D)

    def rows(x):  # and back
        x = x.view(B, N, Hkv, G, C, D).permute(0, 1, 4, 2, 3, 5).reshape(B, N * C, Hq, D)
        return x[:, :Lq].contiguous()

    M = key.shape[2]
    k, v = k.float().transpose(2, 3).contiguous(), v.float().transpose(2, 3).contiguous()  # (B, N, Hkv, M, D)
    q = blocks(s["q"])
    sc = torch.matmul(q, k.transpose(3, 4).contiguous()).mul_(s["scale"]).view(B, N, Hkv, G, C, M)
    sc.masked_fill_(~seen, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    P = sc.sub_(top).exp_()
    total = P.sum(-1, keepdim=True)
    P = P.div_(torch.where(total == 0, 1.0, total)).view(B, N, Hkv, G * C, M)
    o = torch.matmul(P, v)
    out = rows(o).to(t)
    if case["form"] != "train":
        return out
    do = blocks(s["dout"])
    delta = (do * o).sum(-1, keepdim=True)
    dv = torch.matmul(P.transpose(3, 4).contiguous(), do)
    dS = torch.matmul(do, v.transpose(3, 4).contiguous()).sub_(delta).mul_(P).mul_(s["scale"])
    dq = rows(torch.matmul(dS, k)).to(t)
    dk = torch.matmul(dS.transpose(3, 4).contiguous(), q)
    to = (batch * case["Lk"] + at).reshape(-1)

    def gathered(x):  # sums of what each key got from the blocks
        x = x.transpose(2, 3).reshape(-1, Hkv * D)
        return torch.zeros(B * case["Lk"], Hkv * D, device=dev).index_add_(0, to, x).view(B, case["Lk"], Hkv, D).to(t)

    return out, dq, gathered(dk), gathered(dv)


def _plain_recurrence(q, k, v, g, state):
    """o_t = q_t S_t of S_t = exp(g) S_(t-1) + k_t v_t^T over (B, H, L, D) in
    chunks of C: the products inside a chunk, and the states before each."""
    B, H, L, Dk = q.shape
    Dv, dev, C = v.shape[3], q.device, 128
    N = -(-L // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, N * C - L)).view(B, H, N, C, -1) for x in (q, k, v))
    i = torch.arange(C, device=dev, dtype=torch.float32)
    gap = i.view(C, 1) - i.view(1, C)
    inside = torch.where(gap >= 0, torch.exp(g.view(H, 1, 1) * gap.clamp(min=0)), 0.0).view(1, H, 1, C, C)
    o = torch.matmul(torch.matmul(q, k.transpose(3, 4).contiguous()) * inside, v)
    new = torch.matmul((k * torch.exp(g.view(H, 1) * (C - 1 - i)).view(1, H, 1, C, 1)).transpose(3, 4).contiguous(), v)
    n = torch.arange(N, device=dev, dtype=torch.float32)
    gap = n.view(N, 1) - 1 - n.view(1, N)
    across = torch.where(gap >= 0, torch.exp(g.view(H, 1, 1) * C * gap.clamp(min=0)), 0.0).view(1, H, N, N)
    before = torch.matmul(across, new.view(B, H, N, Dk * Dv)).view(B, H, N, Dk, Dv)
    if state is not None:
        before = before + torch.exp(g.view(H, 1) * C * n).view(1, H, N, 1, 1) * state.unsqueeze(2)
    o = o + torch.exp(g.view(H, 1) * (i + 1)).view(1, H, 1, C, 1) * torch.matmul(q, before)
    return o.view(B, H, N * C, Dv)[:, :, :L]


def _plain_linear(s):
    case, t, g = s["case"], s["q"].dtype, s["log_decay"]
    if case["form"] == "step":
        S = s["state"].mul_(torch.exp(g).view(1, -1, 1, 1)).add_(s["k"].float().unsqueeze(3) * s["v"].float().unsqueeze(2))
        o = torch.matmul(s["q"].float().unsqueeze(2), S).squeeze(2) * s["scale"]
        return o.to(t), S
    B, L, H, Dk = s["q"].shape
    token = torch.arange(L, device=g.device)
    lens = torch.full((B,), L, device=g.device) if s["lens"] is None else s["lens"].long()
    there = (token < lens.view(B, 1)).view(B, 1, L, 1)
    # What is past the end is zero, in and out.
    q, k, v = (torch.where(there, s[x].float().transpose(1, 2), 0.0) for x in ("q", "k", "v"))
    given = lambda x: x.transpose(1, 2).to(t).contiguous()  # noqa: E731
    if case["form"] == "prompt":
        out = given(_plain_recurrence(q, k, v, g, s["state"]) * s["scale"])
        left = (lens.view(B, 1, 1) - 1 - token).clamp(min=0).float() * g.view(1, H, 1)
        S = torch.matmul((k * torch.exp(left).unsqueeze(3)).transpose(2, 3).contiguous(), v)
        return out, S + torch.exp(lens.view(B, 1).float() * g).view(B, H, 1, 1) * s["state"]
    do = torch.where(there, s["dout"].float().transpose(1, 2), 0.0)
    back = lambda *x: _plain_recurrence(*(y.flip(2) for y in x), g, None).flip(2) * s["scale"]  # noqa: E731
    out = _plain_recurrence(q, k, v, g, None) * s["scale"]
    dq = _plain_recurrence(do, v, k, g, None) * s["scale"]
    dk, dv = back(v, do, q), back(k, q, do)
    return tuple(given(torch.where(there, x, 0.0)) for x in (out, dq, dk, dv))


# ---- the definition in 64 bits -----------------------------------------------
def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    return (_exact_window if case["op"] == "window" else _exact_linear)(s)


def _exact_window(s):
    """One head at a time, some rows at a time, against every key."""
    case = s["case"]
    B, Lq, Hq, D = s["q"].shape
    Hkv, Lk, W, dev = case["Hkv"], case["Lk"], case["window"], s["q"].device
    nk = _lengths(case, Lk)
    out = torch.zeros(B, Lq, Hq, D, dtype=torch.float64, device=dev)
    train = case["form"] == "train"
    dq = torch.zeros_like(out)
    dk, dv = (torch.zeros(B, Lk, Hkv, D, dtype=torch.float64, device=dev) for _ in range(2))
    for b in range(B):
        n, m = nk[b], min(Lq, nk[b])
        if s["pages"] is None:
            kb, vb = s["k"][b, :n], s["v"][b, :n]
        else:
            kb, vb = (s[x][s["pages"][b].long()].flatten(0, 1)[:n] for x in ("k", "v"))
        j = torch.arange(n, device=dev).view(1, n)
        for h in range(Hq):
            k, v = kb[:, h // (Hq // Hkv)].double(), vb[:, h // (Hq // Hkv)].double()
            for r in range(0, m, 2048):
                e = min(m, r + 2048)
                p = (n - m + torch.arange(r, e, device=dev)).view(-1, 1)
                hidden = (j > p) | ((j <= p - W) & (j >= case["sinks"]))
                q = s["q"][b, r:e, h].double()
                a = torch.softmax((q @ k.T * s["scale"]).masked_fill(hidden, -math.inf), 1)
                o = a @ v
                out[b, r:e, h] = o
                if train:
                    d = s["dout"][b, r:e, h].double()
                    dv[b, :n, h // (Hq // Hkv)] += a.T @ d
                    ds = a * (d @ v.T - (d * o).sum(1, keepdim=True)) * s["scale"]
                    dq[b, r:e, h] = ds @ k
                    dk[b, :n, h // (Hq // Hkv)] += ds.T @ q
    return (out, dq, dk, dv) if train else out


def _exact_linear(s):
    """Every pair of tokens, one head at a time; single tokens by the recurrence."""
    case, g = s["case"], s["log_decay"].double()
    if case["form"] == "step":
        S = torch.exp(g).view(1, -1, 1, 1) * s["state"].double() + torch.einsum("bhk,bhv->bhkv", s["k"].double(), s["v"].double())
        return torch.einsum("bhk,bhkv->bhv", s["q"].double(), S) * s["scale"], S
    B, L, H, Dk = s["q"].shape
    Dv, train = case["Dv"], case["form"] == "train"
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=g.device)  # noqa: E731
    out, dq, dk, dv, S = new(B, L, H, Dv), new(B, L, H, Dk), new(B, L, H, Dk), new(B, L, H, Dv), new(B, H, Dk, Dv)
    for b, n in enumerate(_lengths(case, L)):
        j = torch.arange(n, dtype=torch.float64, device=g.device).view(1, n)
        for h in range(H):
            q, k, v = (s[x][b, :n, h].double() for x in ("q", "k", "v"))
            for r in range(0, n, 2048):
                e = min(n, r + 2048)
                i = j[0, r:e].view(-1, 1)
                fall = torch.exp(g[h] * (i - j).clamp(min=0)).masked_fill(j > i, 0.0) * s["scale"]
                a = (q[r:e] @ k.T) * fall
                out[b, r:e, h] = a @ v
                if train:
                    d = s["dout"][b, r:e, h].double()
                    dv[b, :n, h] += a.T @ d
                    a = (d @ v.T) * fall
                    dq[b, r:e, h] = a @ k
                    dk[b, :n, h] += a.T @ q[r:e]
                else:
                    out[b, r:e, h] += torch.exp(g[h] * (i + 1)) * s["scale"] * (q[r:e] @ s["state"][b, h].double())
            if not train:
                S[b, h] = (k * torch.exp(g[h] * (n - 1 - j)).T).T @ v + torch.exp(g[h] * n) * s["state"][b, h].double()
    return (out, dq, dk, dv) if train else (out, S)
