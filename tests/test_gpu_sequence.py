"""Window attention and linear attention on the GPU against their definitions
in 64 bits (seq_oracle).

Bounds, with u half a step of the element type and A the sum of the absolute
terms of a value: each product that reaches a matrix operand is rounded once
(u A, for linear outputs u A for the products or decayed values and u A for the
state), the result once (u |x|), and 32-bit arithmetic with its exponentials
stays below 2^-13 A. The backward pass of attention reads the rounded output,
which moves delta by u sum |dout out|, inside A as the oracle forms it."""
import math

import pytest
import torch

import memory_efficient_im2win_amd as m
import seq_oracle as O
from parity import device, note

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


def _randn(*shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _bound(r, name, dtype, roundings=1):
    u = O.unit(dtype)
    return (roundings * u + 2.0 ** -13) * r[name + "_abs"] + u * r[name].abs() + 2.0 ** -24


def _ints(x, dev):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)


# B, Lq, Lk, Hq, Hkv, D, window, sinks, q_lens, kv_lens
ATTENTION = [
    (1, 1, 1, 1, 1, 64, 1, 0, None, None),
    (2, 65, 65, 4, 2, 64, 16, 4, None, None),
    (1, 130, 130, 6, 2, 128, 33, 5, None, None),
    (1, 64, 64, 1, 1, 96, 64, 0, None, None),
    (2, 200, 200, 3, 3, 80, 1, 1, None, None),
    (1, 129, 129, 8, 1, 128, 1000, 0, None, None),
    (1, 257, 257, 2, 1, 64, 100, 70, None, None),
    (1, 300, 300, 5, 1, 8, 65, 200, None, None),
    (1, 200, 200, 2, 2, 72, 64, 64, None, None),
    (3, 90, 150, 4, 2, 64, 40, 7, [90, 13, 1], [150, 77, 1]),
    (3, 40, 60, 2, 1, 128, 20, 3, [40, 0, 30], [10, 30, 0]),
    (2, 17, 700, 8, 2, 128, 129, 4, None, [700, 350]),
    (4, 1, 513, 8, 1, 128, 200, 33, None, [513, 200, 1, 0]),
    (2, 3, 400, 2, 2, 40, 400, 0, None, None),
    (1, 1, 3000, 4, 4, 64, 2500, 16, None, None),
]


def _attention_inputs(c, dtype, dev, seed=0):
    B, Lq, Lk, Hq, Hkv, D, window, sinks, ql, kl = c
    q = _randn(B, Lq, Hq, D, dtype=dtype, seed=seed + 1, std=1.5)
    k, v = (_randn(B, Lk, Hkv, D, dtype=dtype, seed=seed + s) for s in (2, 3))
    return q, k, v, dict(window=window, sinks=sinks, scale=D ** -0.5), ql, kl


def _poison(x, lens, value=math.nan):
    """NaN past each sequence's end."""
    x = x.clone()
    for b, n in enumerate(lens or []):
        x[b, max(0, n):] = value
    return x


def _check_forward(out, lse, r, dtype, what):
    O.assert_close(out, r["out"], _bound(r, "out", dtype), what + " out")
    got, want = lse.double().cpu(), r["lse"]
    empty = want == -math.inf
    assert bool((got[empty] == -math.inf).all()), what
    O.assert_close(got[~empty], want[~empty], 1e-5 + 1e-5 * want[~empty].abs(), what + " lse")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("c", ATTENTION, ids=str)
def test_attention(c, dtype):
    dev = device()
    q, k, v, args, ql, kl = _attention_inputs(c, dtype, dev)
    r = O.attention(q, k, v, q_lens=ql, kv_lens=kl, **args)
    note(f"window_attention {c} {dtype}")
    x = [_poison(t, l).to(dev) for t, l in ((q, ql), (k, kl), (v, kl))]
    out, lse = m.window_attention(*x, q_lens=_ints(ql, dev), kv_lens=_ints(kl, dev), return_lse=True, **args)
    torch.cuda.synchronize()
    _check_forward(out, lse, r, dtype, str(c))
    again = m.window_attention(*x, q_lens=_ints(ql, dev), kv_lens=_ints(kl, dev), **args)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("c", ATTENTION, ids=str)
def test_attention_backward(c, dtype):
    dev = device()
    q, k, v, args, ql, kl = _attention_inputs(c, dtype, dev, seed=10)
    dout = _randn(*q.shape, dtype=dtype, seed=9)
    r = O.attention(q, k, v, q_lens=ql, kv_lens=kl, dout=dout, **args)
    lens = dict(q_lens=_ints(ql, dev), kv_lens=_ints(kl, dev))
    note(f"window_attention_backward {c} {dtype}")
    x = [_poison(t, l).to(dev) for t, l in ((q, ql), (k, kl), (v, kl))]
    do = _poison(dout, ql).to(dev)
    out, lse = m.window_attention(*x, return_lse=True, **lens, **args)
    grads = m.window_attention_backward(do, *x, out, lse, **lens, **args)
    torch.cuda.synchronize()
    for n, g in zip(("dq", "dk", "dv"), grads):
        # dq and dk: the rounding of dS, and that of `out` inside delta.
        O.assert_close(g, r[n], _bound(r, n, dtype, 2 if n != "dv" else 1), f"{c} {n}")
    again = m.window_attention_backward(do, *x, out, lse, **lens, **args)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_attention_scales(scale):
    dev = device()
    c = (1, 100, 100, 2, 1, 64, 30, 4, None, None)
    q, k, v, args, _, _ = _attention_inputs(c, torch.bfloat16, dev, seed=20)
    args["scale"] = scale
    dout = _randn(*q.shape, dtype=q.dtype, seed=29)
    r = O.attention(q, k, v, dout=dout, **args)
    note(f"window_attention scale {scale}")
    x = [t.to(dev) for t in (q, k, v)]
    out, lse = m.window_attention(*x, return_lse=True, **args)
    grads = m.window_attention_backward(dout.to(dev), *x, out, lse, **args)
    torch.cuda.synchronize()
    _check_forward(out, lse, r, q.dtype, f"scale {scale}")
    for n, g in zip(("dq", "dk", "dv"), grads):
        O.assert_close(g, r[n], _bound(r, n, q.dtype, 2), f"scale {scale} {n}")


# page, B, Lq, Lk, Hq, Hkv, D, window, sinks, q_lens, kv_lens
PAGED = [
    (16, 3, 1, 640, 8, 2, 128, 100, 17, None, [640, 301, 5]),
    (64, 2, 1, 4096, 4, 4, 64, 2000, 4, None, [4000, 77]),
    (16, 2, 50, 336, 6, 2, 80, 64, 3, [50, 20], [330, 21]),
    (7, 2, 5, 210, 4, 1, 96, 40, 9, [5, 5], [203, 100]),
    (1, 1, 3, 130, 2, 1, 64, 70, 2, None, [129]),
    (256, 1, 1, 512, 2, 1, 128, 300, 0, None, [500]),
]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("c", PAGED, ids=str)
def test_attention_over_pages(c, dtype):
    """Pages in a mixed order. Pages that no query sees are gone (-1 and far
    past the pool in turn), pages without an owner and what lies past the
    lengths or before the windows hold NaN."""
    page, *c = c
    dev = device()
    B, Lq, Lk, Hq, Hkv, D, window, sinks, ql, kl = c
    q, k, v, args, _, _ = _attention_inputs(c, dtype, dev, seed=30)
    r = O.attention(q, k, v, q_lens=ql, kv_lens=kl, **args)
    per = Lk // page
    pages = B * per + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(5))[:B * per].view(B, per)
    pk = torch.full((pages, page, Hkv, D), math.nan, dtype=dtype)
    pv = pk.clone()
    table = order.to(torch.int32)
    for b, (mq, n) in enumerate(zip(O.lengths(ql, B, Lq), O.lengths(kl, B, Lk))):
        used = torch.zeros(Lk, dtype=torch.bool)
        used[:n] = O.visible(mq, n, window, sinks).any(0)
        for j in used.nonzero().view(-1).tolist():
            pk[order[b, j // page], j % page] = k[b, j]
            pv[order[b, j // page], j % page] = v[b, j]
        for t in range(per):
            if not used[t * page:(t + 1) * page].any():
                table[b, t] = -1 if t % 2 else 2**31 - 1
    note(f"window_attention over pages {c} page {page} {dtype}")
    out, lse = m.window_attention(q.to(dev), pk.to(dev), pv.to(dev), q_lens=_ints(ql, dev), kv_lens=_ints(kl, dev),
                                  page_table=table.to(dev), return_lse=True, **args)
    torch.cuda.synchronize()
    _check_forward(out, lse, r, dtype, str(c))


def test_a_page_outside_the_pool_is_nan():
    dev = device()
    x = _randn(4, 16, 1, 64, dtype=torch.bfloat16, seed=1).to(dev)
    q = _randn(2, 1, 2, 64, dtype=torch.bfloat16, seed=2).to(dev)
    for bad in (-1, 4, 2**31 - 1):
        table = torch.tensor([[0, bad], [2, 3]], dtype=torch.int32, device=dev)
        note(f"page {bad} of 4")
        out = m.window_attention(q, x, x, window=20, page_table=table).float().cpu()
        assert bool(out[0].isnan().all()) and bool(out[1].isfinite().all())


def test_attention_over_a_cache_past_32_bits():
    """Pages whose offsets pass 2^31 and 2^32 elements."""
    dev = device()
    page, Hkv, D, Hq, n = 64, 8, 128, 16, 300
    per_page = page * Hkv * D
    pages = (1 << 32) // per_page + 9
    pool = torch.empty(2, pages, page, Hkv, D, dtype=torch.bfloat16, device=dev)
    ids = [pages - 1, (1 << 31) // per_page + 1, 3, (1 << 31) // per_page - 1, pages - 5]
    k, v = (_randn(1, 5 * page, Hkv, D, dtype=torch.bfloat16, seed=s) for s in (1, 2))
    for t, p in enumerate(ids):
        pool[0, p] = k[0, t * page:(t + 1) * page].to(dev)
        pool[1, p] = v[0, t * page:(t + 1) * page].to(dev)
    q = _randn(1, 2, Hq, D, dtype=torch.bfloat16, seed=3)
    r = O.attention(q, k, v, 200, 70, 0.1, None, [n])
    note("cache past 32 bits")
    out = m.window_attention(q.to(dev), pool[0], pool[1], window=200, sinks=70, scale=0.1,
                             kv_lens=_ints([n], dev), page_table=_ints([ids], dev))
    torch.cuda.synchronize()
    O.assert_close(out, r["out"], _bound(r, "out", q.dtype), "far pages")


def test_attention_strides():
    """One projection's parts, heads before tokens, a batch that shares its
    keys, and outputs with strides of their own."""
    dev = device()
    dtype = torch.float16
    B, L, Hq, Hkv, D = 2, 75, 4, 2, 64
    x = _randn(B, L, (Hq + 2 * Hkv) * D, dtype=dtype, seed=1).to(dev)
    q, k, v = (y.unflatten(2, (-1, D)) for y in x.split([Hq * D, Hkv * D, Hkv * D], 2))
    k = k[:1].expand(B, L, Hkv, D)
    v = v.transpose(1, 2).contiguous().transpose(1, 2)
    dout = _randn(B, L, Hq, D + 8, dtype=dtype, seed=2).to(dev)[..., :D]
    args = dict(window=20, sinks=3, scale=0.2)
    r = O.attention(q, k, v, dout=dout, **args)
    room = torch.full((B, Hq, L, D + 16), 7.0, dtype=dtype, device=dev)
    out = room[..., 8:8 + D].transpose(1, 2)
    note("window_attention strides")
    res, lse = m.window_attention(q, k, v, out=out, return_lse=True, **args)
    dqkv = torch.full_like(x, 5.0)
    dq, _, dv = (y.unflatten(2, (-1, D)) for y in dqkv.split([Hq * D, Hkv * D, Hkv * D], 2))
    got = m.window_attention_backward(dout, q, k, v, out, lse, dq=dq, dv=dv, **args)
    torch.cuda.synchronize()
    assert res is out and got[0] is dq and got[2] is dv
    _check_forward(out, lse, r, dtype, "strides")
    for n, g in zip(("dq", "dk", "dv"), got):
        O.assert_close(g, r[n], _bound(r, n, dtype, 2), f"strides {n}")
    assert bool((room[..., :8] == 7).all()) and bool((room[..., 8 + D:] == 7).all())
    assert bool((dqkv[..., Hq * D:(Hq + Hkv) * D] == 5).all())


def test_lengths_out_of_range_are_cut():
    dev = device()
    q, k, v, args, _, _ = _attention_inputs((3, 20, 40, 2, 1, 64, 10, 2, None, None), torch.bfloat16, dev, seed=40)
    r = O.attention(q, k, v, q_lens=[20, 0, 20], kv_lens=[40, 40, 0], **args)
    note("lengths out of range")
    x = [t.to(dev) for t in (q, k, v)]
    out, lse = m.window_attention(*x, q_lens=_ints([1000, -5, 20], dev), kv_lens=_ints([2**31 - 1, 40, -1], dev),
                                  return_lse=True, **args)
    torch.cuda.synchronize()
    _check_forward(out, lse, r, q.dtype, "cut lengths")


def test_attention_of_empty_tensors():
    dev = device()
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device=dev)  # noqa: E731
    assert m.window_attention(z(0, 4, 2, 64), z(0, 4, 1, 64), z(0, 4, 1, 64), window=2).shape == (0, 4, 2, 64)
    assert m.window_attention(z(2, 0, 2, 64), z(2, 4, 1, 64), z(2, 4, 1, 64), window=2).shape == (2, 0, 2, 64)
    q = torch.ones(2, 3, 2, 64, dtype=torch.float16, device=dev)
    out, lse = m.window_attention(q, z(2, 0, 1, 64), z(2, 0, 1, 64), window=2, return_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())
    dq, dk, dv = m.window_attention_backward(q, q, z(2, 0, 1, 64), z(2, 0, 1, 64), out, lse, window=2)
    assert not dq.any() and dk.shape == dv.shape == (2, 0, 1, 64)


# B, L, H, Dk, Dv, lens, log decays
LINEAR = [
    (1, 1, 1, 64, 64, None, [-0.1]),
    (2, 31, 2, 64, 128, None, [0.0, -0.5]),
    (1, 32, 1, 128, 64, None, [-0.01]),
    (1, 33, 3, 96, 80, None, [-3.0, -0.2, -1e-3]),
    (3, 130, 2, 128, 128, [130, 64, 0], [-0.03, -math.inf]),
    (2, 200, 2, 8, 40, [1, 129], [-0.004, -200.0]),
    (1, 500, 1, 128, 96, None, [-0.004]),
    (2, 257, 5, 72, 16, None, [-0.7, -0.1, -0.02, -0.004, 0.0]),
]


def _linear_inputs(c, dtype, seed=0):
    B, L, H, Dk, Dv, lens, g = c
    q, k = (_randn(B, L, H, Dk, dtype=dtype, seed=seed + s) for s in (1, 2))
    v = _randn(B, L, H, Dv, dtype=dtype, seed=seed + 3)
    state = _randn(B, H, Dk, Dv, dtype=torch.float32, seed=seed + 4, std=2.0)
    return q, k, v, torch.tensor(g, dtype=torch.float32), state, lens


def _state_bound(r, name):
    # 22 bits or more of every decayed value, 32-bit sums.
    return 2.0 ** -17 * r[name + "_abs"] + 2.0 ** -22


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("c", LINEAR, ids=str)
def test_linear(c, dtype, given):
    dev = device()
    q, k, v, g, state, lens = _linear_inputs(c, dtype)
    scale = 0.11
    r = O.linear(q, k, v, g, scale, state if given else None, lens)
    note(f"linear_attention {c} {dtype} state {given}")
    x = [_poison(t, lens).to(dev) for t in (q, k, v)]
    out, s = m.linear_attention(*x, g.to(dev), state=state.to(dev) if given else None, scale=scale,
                                lens=_ints(lens, dev))
    torch.cuda.synchronize()
    O.assert_close(out, r["out"], _bound(r, "out", dtype, 2), f"{c} out")
    O.assert_close(s, r["state"], _state_bound(r, "state"), f"{c} state")
    again = m.linear_attention(*x, g.to(dev), state=state.to(dev) if given else None, scale=scale,
                               lens=_ints(lens, dev))
    assert torch.equal(out, again[0]) and torch.equal(s, again[1])


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("c", LINEAR, ids=str)
def test_linear_backward(c, dtype, given):
    dev = device()
    q, k, v, g, state, lens = _linear_inputs(c, dtype, seed=10)
    dout = _randn(*v.shape, dtype=dtype, seed=19)
    dstate = _randn(*state.shape, dtype=torch.float32, seed=18)
    scale = 0.11
    r = O.linear(q, k, v, g, scale, state if given else None, lens, dout, dstate if given else None)
    note(f"linear_attention_backward {c} {dtype} state {given}")
    x = [_poison(t, lens).to(dev) for t in (dout, q, k, v)]
    args = dict(scale=scale, lens=_ints(lens, dev))
    if given:
        args.update(state=state.to(dev), dstate=dstate.to(dev))
    got = m.linear_attention_backward(*x, g.to(dev), **args)
    torch.cuda.synchronize()
    for n, y in zip(("dq", "dk", "dv"), got):
        O.assert_close(y, r[n], _bound(r, n, dtype, 2), f"{c} {n}")
    assert (got[3] is not None) == given
    if given:
        O.assert_close(got[3], r["dstate"], _state_bound(r, "dstate"), f"{c} dstate")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("c", [(1, 1, 64, 64), (3, 5, 128, 128), (2, 7, 96, 80), (70, 8, 64, 128), (1, 3, 8, 16),
                               (2, 2, 128, 8)], ids=str)
def test_linear_step(c, dtype):
    dev = device()
    B, H, Dk, Dv = c
    g = -torch.logspace(-3, 1, H)
    q, k, v, _, state, _ = _linear_inputs((B, 3, H, Dk, Dv, None, g.tolist()), dtype, seed=50)
    r = O.linear(q, k, v, g, 0.2, state)
    note(f"linear_attention_step {c} {dtype}")
    s = state.to(dev)
    for t in range(3):
        out = m.linear_attention_step(*(x[:, t].to(dev) for x in (q, k, v)), g.to(dev), s, scale=0.2)
        want = {"x": r["out"][:, t], "x_abs": r["out_abs"][:, t]}
        O.assert_close(out, want["x"], _bound(want, "x", dtype, 0), f"{c} token {t}")
    # All in 32 bits: three decays, products and sums.
    O.assert_close(s, r["state"], 2.0 ** -20 * r["state_abs"], f"{c} state")


def test_prompt_then_steps_is_the_whole():
    """A prompt in two calls, the second over lengths, then single tokens."""
    dev = device()
    c = (2, 150, 3, 64, 80, None, [-0.5, -0.03, 0.0])
    q, k, v, g, state, _ = _linear_inputs(c, torch.bfloat16, seed=60)
    r = O.linear(q, k, v, g, 0.125, state)
    x = [t.to(dev) for t in (q, k, v)]
    note("prompt, then steps")
    s = state.to(dev)
    a, s2 = m.linear_attention(*(t[:, :70] for t in x), g.to(dev), state=s, state_out=s, scale=0.125)
    assert s2 is s
    b, _ = m.linear_attention(*(t[:, 70:] for t in x), g.to(dev), state=s, state_out=s, scale=0.125,
                              lens=_ints([75, 75], dev))
    outs = [a, b[:, :75]]
    for t in range(145, 150):
        outs.append(m.linear_attention_step(*(y[:, t] for y in x), g.to(dev), s, scale=0.125).unsqueeze(1))
    torch.cuda.synchronize()
    O.assert_close(torch.cat(outs, 1), r["out"], _bound(r, "out", q.dtype, 2), "out")
    O.assert_close(s, r["state"], _state_bound(r, "state"), "state")


def test_linear_strides_and_outputs():
    dev = device()
    dtype = torch.float16
    B, L, H, Dk, Dv = 2, 70, 3, 64, 96
    x = _randn(B, L, H * (2 * Dk + Dv), dtype=dtype, seed=1).to(dev)
    q, k, v = (y.unflatten(2, (H, -1)) for y in x.split([H * Dk, H * Dk, H * Dv], 2))
    v = v.transpose(1, 2).contiguous().transpose(1, 2)
    g = torch.tensor([-0.1, -0.01, -1.0])
    r = O.linear(q, k, v, g, 0.3)
    room = torch.full((B, H, L, Dv + 8), 7.0, dtype=dtype, device=dev)
    note("linear_attention strides")
    out, s = m.linear_attention(q, k, v, g.to(dev), scale=0.3, out=room[..., :Dv].transpose(1, 2))
    torch.cuda.synchronize()
    O.assert_close(out, r["out"], _bound(r, "out", dtype, 2), "out")
    O.assert_close(s, r["state"], _state_bound(r, "state"), "state")
    assert bool((room[..., Dv:] == 7).all())


def test_linear_of_no_tokens_keeps_the_state():
    dev = device()
    state = torch.randn(2, 3, 64, 64, device=dev)
    z = torch.zeros(2, 0, 3, 64, dtype=torch.float16, device=dev)
    out, s = m.linear_attention(z, z, z, torch.full((3,), -0.5, device=dev), state=state)
    assert out.shape == (2, 0, 3, 64) and torch.equal(s, state)


def test_other_streams_and_given_workspaces():
    dev = device()
    q, k, v, args, _, _ = _attention_inputs((1, 5, 900, 4, 2, 64, 800, 4, None, None), torch.bfloat16, dev, seed=70)
    x = [t.to(dev) for t in (q, k, v)]
    g = torch.tensor([-0.1, -0.02], device=dev)
    want = m.window_attention(*x, **args), m.linear_attention(x[1], x[1], x[2], g)[0]
    torch.cuda.synchronize()
    note("another stream, own workspaces")
    side = torch.cuda.Stream()
    ws = torch.empty(max(m.window_attention_workspace_bytes(1, 5, 900, 4, 2, 64, 800, 4),
                         m.linear_attention_workspace_bytes(1, 900, 2, 64, 64)), dtype=torch.uint8, device=dev)
    with torch.cuda.stream(side):
        a = m.window_attention(*x, ws=ws, **args)
        b = m.linear_attention(x[1], x[1], x[2], g, ws=ws)[0]
    side.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    with pytest.raises(m.Im2winError):
        m.window_attention(*x, ws=ws[:16], **args)


def test_calls_in_a_graph():
    """Captured once, replayed over new inputs with eager work in between."""
    dev = device()
    q, k, v, args, _, _ = _attention_inputs((1, 40, 600, 4, 2, 64, 500, 4, None, None), torch.float16, dev, seed=80)
    x = [t.to(dev) for t in (q, k, v)]
    dout = torch.randn(q.shape, device=dev).half()
    g = torch.tensor([-0.1, -0.02], device=dev)
    state = torch.zeros(1, 2, 64, 64, device=dev)

    def work(s):
        out, lse = m.window_attention(*x, return_lse=True, **args)
        grads = m.window_attention_backward(dout, *x, out, lse, **args)
        y, _ = m.linear_attention(x[1], x[1], x[2], g, state=s)
        back = m.linear_attention_backward(y, x[1], x[1], x[2], g)
        step = m.linear_attention_step(x[1][:, 0], x[1][:, 1], x[2][:, 2], g, s)
        return [out, *grads, y, *back[:3], step, s]

    work(state.clone())
    torch.cuda.synchronize()
    note("graph capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work(state)
    for i in range(4):
        for t, s in zip(x, (1.5, 1.0, 1.0)):
            t.copy_((torch.randn(t.shape, device=dev) * s).half())
        state.normal_()
        begin = state.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = work(begin)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_binding_refuses():
    dev = device()
    z = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype, device=dev)  # noqa: E731
    q, k = z(1, 4, 4, 64), z(1, 8, 2, 64)
    g, st = torch.zeros(2, device=dev), torch.zeros(1, 2, 64, 64, device=dev)
    W, LA = m.window_attention, m.linear_attention
    for err, call in [
        (TypeError, lambda: W(q.float(), k.float(), k.float(), window=2)),
        (TypeError, lambda: W(q, k.bfloat16(), k, window=2)),
        (ValueError, lambda: W(q, k, k, window=0)),
        (ValueError, lambda: W(q, k, k, window=2, sinks=-1)),
        (ValueError, lambda: W(q, k, k, window=2, scale=math.inf)),
        (ValueError, lambda: W(q[:, :, :3], k, k, window=2)),
        (ValueError, lambda: W(q[..., :60], k[..., :60], k[..., :60], window=2)),
        (ValueError, lambda: W(z(1, 4, 4, 136), z(1, 4, 4, 136), z(1, 4, 4, 136), window=2)),
        (ValueError, lambda: W(q, k, k[:, :7], window=2)),
        (ValueError, lambda: W(q, k.cpu(), k, window=2)),
        (ValueError, lambda: W(z(1, 4, 4, 68)[..., :64], k, k, window=2)),
        (ValueError, lambda: W(q.transpose(2, 3).contiguous().transpose(2, 3), k, k, window=2)),
        (ValueError, lambda: W(q, k, k, window=2, kv_lens=torch.zeros(1, dtype=torch.int64, device=dev))),
        (ValueError, lambda: W(q, k, k, window=2, kv_lens=torch.zeros(2, dtype=torch.int32, device=dev))),
        (ValueError, lambda: W(q, k, k, window=2, q_lens=torch.zeros(1, dtype=torch.int32))),
        (ValueError, lambda: W(q, k, k, window=2, page_table=torch.zeros(2, 1, dtype=torch.int32, device=dev))),
        (ValueError, lambda: W(q, k, k, window=2, out=z(1, 4, 4, 32))),
        (ValueError, lambda: W(q, k, k, window=2, out=z(1, 1, 4, 64).expand(1, 4, 4, 64))),
        (ValueError, lambda: m.window_attention_backward(q, q, k, k, q, None, window=2)),
        (ValueError, lambda: m.window_attention_backward(q, q, k, k, q, torch.zeros(1, 4, 5, device=dev), window=2)),
        (TypeError, lambda: LA(k.float(), k.float(), k.float(), g)),
        (ValueError, lambda: LA(k, k, k, torch.zeros(3, device=dev))),
        (ValueError, lambda: LA(k, k, k, g.double())),
        (ValueError, lambda: LA(k, k, k, None)),
        (ValueError, lambda: LA(k, k, k[:, :7], g)),
        (ValueError, lambda: LA(k, k, k, g, state=st.half())),
        (ValueError, lambda: LA(k, k, k, g, state=st.transpose(2, 3))),
        (ValueError, lambda: m.linear_attention_step(k[:, 0], k[:, 1], k[:, 2], g, None)),
        (ValueError, lambda: m.linear_attention_step(k, k, k, g, st)),
    ]:
        with pytest.raises(err):
            call()
