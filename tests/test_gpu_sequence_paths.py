"""The ways that sequence operators take by size and layout, against their
definitions in 64 bits, and the example that runs them together. The bounds are
those of test_gpu_sequence.py: u A for each rounded operand (u: half a step of
the type, A: the sum of a value's absolute terms), u |x| for the result,
2^-13 A for 32-bit arithmetic, 2^-17 A for states."""
import importlib.util
import math
import os

import pytest
import torch

import memory_efficient_im2win_amd as m
import seq_oracle as O
from parity import device, note
from test_gpu_sequence import TYPES, _bound, _check_forward, _ints, _linear_inputs, _poison, _randn, _state_bound

pytestmark = pytest.mark.gpu


# Sequences of a few segments, with the last state apart from the first one and
# in its place.
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("state_given", ["none", "apart", "replaced"])
@pytest.mark.parametrize("c", [
    (2, 200, 2, 64, 64, [200, 70], [-0.02, 0.0]),
    (1, 300, 3, 128, 128, None, [-0.7, -0.01, -math.inf]),
    (2, 140, 1, 96, 40, [0, 139], [-1e-3]),
    (1, 129, 2, 64, 128, [97], [-0.05, -0.3]),
], ids=str)
def test_linear_of_few_segments(c, state_given, dtype):
    dev = device()
    q, k, v, g, state, lens = _linear_inputs(c, dtype, seed=60)
    r = O.linear(q, k, v, g, 0.11, None if state_given == "none" else state, lens)
    note(f"linear_attention {c} {dtype} state {state_given}")
    x = [_poison(t, lens).to(dev) for t in (q, k, v)]
    args = dict(scale=0.11, lens=_ints(lens, dev))
    if state_given != "none":
        args["state"] = state.to(dev)
    if state_given == "replaced":
        args["state_out"] = args["state"]
    out, s = m.linear_attention(*x, g.to(dev), **args)
    torch.cuda.synchronize()
    O.assert_close(out, r["out"], _bound(r, "out", dtype, 2), f"{c} out")
    O.assert_close(s, r["state"], _state_bound(r, "state"), f"{c} state")


# Enough rows for workgroups of 128: pages that hold tiles of 64 keys, that hold
# parts of them, and that end inside a copy.
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("page,D", [(64, 128), (192, 64), (16, 80), (8, 128), (7, 72), (1, 64)])
def test_prompts_over_pages(page, D, dtype):
    dev = device()
    B, Lq, Lk, Hq, Hkv, window, sinks = 8, 130, 384, 16, 8, 90, 11
    ql, kl = [130, 130, 64, 1, 130, 0, 99, 130], [384, 131, 200, 77, 130, 50, 99, 60]
    q = _randn(B, Lq, Hq, D, dtype=dtype, seed=71, std=1.5)
    k, v = (_randn(B, Lk, Hkv, D, dtype=dtype, seed=s) for s in (72, 73))
    args = dict(window=window, sinks=sinks, scale=D ** -0.5)
    r = O.attention(q, k, v, q_lens=ql, kv_lens=kl, **args)
    per = -(-Lk // page)
    pages = B * per + 1
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(7))[:B * per].view(B, per)
    pool = torch.full((2, pages * page, Hkv, D), math.nan, dtype=dtype)
    table = order.to(torch.int32)
    slot = (order.unsqueeze(2) * page + torch.arange(page)).flatten(1)[:, :Lk]
    for b in range(B):
        used = torch.zeros(Lk, dtype=torch.bool)
        used[:kl[b]] = O.visible(ql[b], kl[b], window, sinks).any(0)
        at = used.nonzero().view(-1)
        pool[0, slot[b, at]], pool[1, slot[b, at]] = k[b, at], v[b, at]
        for t in range(per):
            if not used[t * page:(t + 1) * page].any():
                table[b, t] = -1 if t % 2 else 2**31 - 1
    pk, pv = (x.view(pages, page, Hkv, D).to(dev) for x in pool)
    note(f"window_attention prompts over pages of {page}, D {D} {dtype}")
    lens = dict(q_lens=_ints(ql, dev), kv_lens=_ints(kl, dev))
    out, lse = m.window_attention(q.to(dev), pk, pv, page_table=table.to(dev), return_lse=True, **lens, **args)
    torch.cuda.synchronize()
    _check_forward(out, lse, r, dtype, f"page {page}")
    # A page outside the pool under the last keys of sequence 0.
    table[0, (kl[0] - 1) // page] = pages
    out = m.window_attention(q.to(dev), pk, pv, page_table=table.to(dev), **lens, **args).cpu()
    assert bool(out[0, -1].isnan().all()) and torch.isfinite(out[1:]).all()


@pytest.mark.parametrize("page", [64, 128, 1])
def test_a_token_over_a_page_outside_the_pool_is_nan(page):
    dev = device()
    x = _randn(4, page, 1, 64, dtype=torch.bfloat16, seed=1).to(dev)
    q = _randn(2, 1, 2, 64, dtype=torch.bfloat16, seed=2).to(dev)
    for bad in (-1, 4, 2**31 - 1):
        table = torch.tensor([[0, bad], [2, 3]], dtype=torch.int32, device=dev)
        note(f"page {bad} of 4, {page} tokens each")
        out = m.window_attention(q, x, x, window=page + 1, page_table=table).float().cpu()
        assert bool(out[0].isnan().all()) and bool(out[1].isfinite().all())


def test_numbers_given_as_tensors_are_read_at_each_call():
    dev = device()
    q, k, v = (_randn(1, 40, 2, 64, dtype=torch.bfloat16, seed=s).to(dev) for s in (1, 2, 3))
    window = torch.tensor(4)
    a = m.window_attention(q, k, v, window=window)
    window.fill_(30)
    b = m.window_attention(q, k, v, window=window)
    assert torch.equal(a, m.window_attention(q, k, v, window=4))
    assert torch.equal(b, m.window_attention(q, k, v, window=30)) and not torch.equal(a, b)


def test_example_decoder():
    """Logits of 4 layers in bfloat16, token by token and as one sequence: the
    same values rounded apart in about 8 places a layer, 32 * 2^-8 at worst."""
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decoder.py")
    spec = importlib.util.spec_from_file_location("hybrid_decoder", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    device()
    note("hybrid decoder")
    off, losses = example.main(["--prompt", "150", "--new", "6", "--steps", "4"])
    assert off < 32 * 2.0 ** -8
    assert losses[-1] < losses[0]
