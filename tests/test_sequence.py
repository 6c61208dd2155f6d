"""The sequence operators on the host: definitions against differences and
autograd, refusals of the C ABI and of the binding (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

import memory_efficient_im2win_amd as m
import seq_oracle as O
from memory_efficient_im2win_amd import _lib, sequence

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every call below fails its checks first


def test_header_and_binding_name_the_same_entry_points():
    text = open(os.path.join(ROOT, "include", "im2win_seq.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(im2win_seq_\w+)\s*\(", text))
    assert names == set(_lib.SEQ_EXPORTS)
    L = m.load_library()
    for n in names:
        assert hasattr(L, n)


# ---- the definitions ---------------------------------------------------------
def _randn(*shape, seed=0):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed))


def test_attention_gradients_are_the_differences():
    B, Lq, Lk, Hq, Hkv, D = 2, 7, 9, 4, 2, 8
    q, k, v = _randn(B, Lq, Hq, D, seed=1), _randn(B, Lk, Hkv, D, seed=2), _randn(B, Lk, Hkv, D, seed=3)
    dout = _randn(B, Lq, Hq, D, seed=4)
    args = dict(window=3, sinks=2, scale=0.4, q_lens=[7, 4], kv_lens=[9, 5])
    r = O.attention(q, k, v, dout=dout, **args)
    loss = lambda *x: (O.attention(*x, **args)["out"] * dout).sum()  # noqa: E731
    for i, name in enumerate(("dq", "dk", "dv")):
        step = _randn(*(q, k, v)[i].shape, seed=5 + i)
        lo, hi = [q, k, v], [q, k, v]
        lo[i], hi[i] = lo[i] - 1e-5 * step, hi[i] + 1e-5 * step
        assert abs((loss(*hi) - loss(*lo)) / 2e-5 - (r[name] * step).sum()) < 1e-7


def test_linear_gradients_are_the_differences():
    B, L, H, Dk, Dv = 2, 6, 3, 8, 16
    x = [_randn(B, L, H, Dk, seed=1), _randn(B, L, H, Dk, seed=2), _randn(B, L, H, Dv, seed=3),
         _randn(B, H, Dk, Dv, seed=4)]
    g = torch.tensor([0.0, -0.1, -2.0], dtype=torch.float64)
    dout, dstate, lens = _randn(B, L, H, Dv, seed=5), _randn(B, H, Dk, Dv, seed=6), [6, 4]
    f = lambda y: O.linear(*y[:3], g, 0.3, y[3], lens)  # noqa: E731

    def loss(y):
        r = f(y)
        return (r["out"] * dout).sum() + (r["state"] * dstate).sum()

    r = O.linear(*x[:3], g, 0.3, x[3], lens, dout, dstate)
    for i, name in enumerate(("dq", "dk", "dv", "dstate")):
        step = _randn(*x[i].shape, seed=7 + i)
        lo = [y - 1e-5 * step if j == i else y for j, y in enumerate(x)]
        hi = [y + 1e-5 * step if j == i else y for j, y in enumerate(x)]
        assert abs((loss(hi) - loss(lo)) / 2e-5 - (r[name] * step).sum()) < 1e-7


def test_step_by_step_attention_is_the_prompt():
    q, k, v = _randn(1, 9, 2, 8, seed=1), _randn(1, 9, 1, 8, seed=2), _randn(1, 9, 1, 8, seed=3)
    whole = O.attention(q, k, v, 3, 2, 0.5)["out"]
    for i in range(9):
        one = O.attention(q[:, i:i + 1], k[:, :i + 1], v[:, :i + 1], 3, 2, 0.5)["out"]
        assert torch.allclose(one[:, 0], whole[:, i], atol=1e-12)


# ---- refusals of the C ABI ---------------------------------------------------
T = (FAKE, 64, 64, 64)  # a tensor: pointer and strides


def _attention(q=T, k=T, v=T, out=T, lse=FAKE, q_lens=0, kv_lens=0, table=0, table_stride=0, dtype=1, B=1, Lq=4, Lk=4,
               Hq=2, Hkv=1, D=64, page=0, pages=0, window=2, sinks=0, scale=1.0, dout=T, dq=T, dk=T, dv=T):
    return sequence._ATTENTION.pack(*q, *k, *v, *out, lse, q_lens, kv_lens, table, table_stride, dtype, B, Lq, Lk, Hq,
                                    Hkv, D, page, pages, window, sinks, scale, *dout, *dq, *dk, *dv)


def _linear(q=T, k=T, v=T, out=T, decay=FAKE, state_in=0, state_out=0, lens=0, dtype=1, B=1, L=4, H=2, Dk=64, Dv=64,
            scale=1.0, dout=T, dq=T, dk=T, dv=T, dstate_out=0, dstate_in=0):
    return sequence._LINEAR.pack(*q, *k, *v, *out, decay, state_in, state_out, lens, dtype, B, L, H, Dk, Dv, scale,
                                 *dout, *dq, *dk, *dv, dstate_out, dstate_in)


BAD_TENSORS = [(0, 64, 64, 64), (FAKE + 8, 64, 64, 64), (FAKE, 60, 64, 64), (FAKE, 64, 4, 64), (FAKE, 64, 64, -64),
               (FAKE, 64, 1 << 24, 64)]
BAD_ATTENTION = ([dict(dtype=2), dict(dtype=-1), dict(B=-1), dict(Lq=-1), dict(Lk=-1), dict(Hq=3, Hkv=2), dict(Hkv=0),
                  dict(Hq=0), dict(D=0), dict(D=12), dict(D=136), dict(window=0), dict(sinks=-1),
                  dict(scale=float("nan")), dict(scale=float("inf")), dict(Lq=1 << 30), dict(Lk=(1 << 30) + 1),
                  dict(lse=FAKE + 2), dict(q_lens=FAKE + 1), dict(kv_lens=FAKE + 2), dict(page=4),
                  dict(B=1 << 30, Lq=64)] + [{n: t} for n in ("q", "k", "v", "out") for t in BAD_TENSORS])


@pytest.mark.parametrize("bad", BAD_ATTENTION, ids=str)
def test_attention_refuses(bad):
    L = m.load_library()
    args = _attention(**bad)
    ws = L.im2win_seq_attention_workspace_bytes(_attention())
    assert L.im2win_seq_attention(args, FAKE, ws, None) == _lib.IM2WIN_EINVAL
    assert L.im2win_seq_attention_backward(args, FAKE, 1 << 40, None) == _lib.IM2WIN_EINVAL
    if not set(bad) & {"q", "k", "v", "out", "lse", "q_lens", "kv_lens"}:
        assert L.im2win_seq_attention_workspace_bytes(args) == 0
        assert L.im2win_seq_attention_backward_workspace_bytes(args) == 0


@pytest.mark.parametrize("bad", [dict(page=0), dict(pages=-1), dict(table=FAKE + 1)], ids=str)
def test_paged_attention_refuses(bad):
    args = _attention(**{**dict(table=FAKE, table_stride=1, page=4, pages=1), **bad})
    assert m.load_library().im2win_seq_attention(args, None, 0, None) == _lib.IM2WIN_EINVAL


def test_attention_backward_refuses():
    L = m.load_library()
    f = L.im2win_seq_attention_backward
    need = L.im2win_seq_attention_backward_workspace_bytes(_attention())
    assert need > 0
    assert f(_attention(), FAKE, need - 1, None) == _lib.IM2WIN_EWORKSPACE
    assert f(_attention(), None, 0, None) == _lib.IM2WIN_EWORKSPACE
    assert f(_attention(), FAKE + 4, need, None) == _lib.IM2WIN_EINVAL
    assert f(_attention(lse=0), FAKE, need, None) == _lib.IM2WIN_EINVAL
    assert f(_attention(table=FAKE, table_stride=1, page=4, pages=1), FAKE, need, None) == _lib.IM2WIN_EINVAL
    for n in ("dout", "dq", "dk", "dv"):
        for t in BAD_TENSORS:
            assert f(_attention(**{n: t}), FAKE, need, None) == _lib.IM2WIN_EINVAL
    assert f(None, FAKE, need, None) == _lib.IM2WIN_EINVAL


def test_workspaces_too_small():
    L = m.load_library()
    one = dict(Lq=1, Lk=8192, window=4096)
    need = L.im2win_seq_attention_workspace_bytes(_attention(**one))
    assert need > 0
    assert L.im2win_seq_attention(_attention(**one), FAKE, need - 1, None) == _lib.IM2WIN_EWORKSPACE
    assert L.im2win_seq_attention(_attention(**one), None, 0, None) == _lib.IM2WIN_EWORKSPACE
    need = L.im2win_seq_linear_workspace_bytes(_linear(L=4096))
    assert need > 0
    assert L.im2win_seq_linear(_linear(L=4096), FAKE, need - 1, None) == _lib.IM2WIN_EWORKSPACE
    need = L.im2win_seq_linear_backward_workspace_bytes(_linear(L=4096))
    assert L.im2win_seq_linear_backward(_linear(L=4096), FAKE, need - 1, None) == _lib.IM2WIN_EWORKSPACE


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(B=-1), dict(L=-1), dict(H=0), dict(Dk=4), dict(Dv=130),
                                 dict(Dk=136), dict(scale=float("nan")), dict(decay=0), dict(decay=FAKE + 1),
                                 dict(lens=FAKE + 2), dict(state_in=FAKE + 4), dict(state_out=FAKE + 4),
                                 dict(L=1 << 30, B=1 << 10)] +
                         [{n: t} for n in ("q", "k", "v", "out") for t in BAD_TENSORS], ids=str)
def test_linear_refuses(bad):
    L = m.load_library()
    args = _linear(**bad)
    assert L.im2win_seq_linear(args, FAKE, 1 << 40, None) == _lib.IM2WIN_EINVAL
    assert L.im2win_seq_linear_step(_linear(**{**dict(L=1, state_in=FAKE, state_out=FAKE), **bad}), None) == \
        _lib.IM2WIN_EINVAL
    if "out" not in bad:
        assert L.im2win_seq_linear_backward(args, FAKE, 1 << 40, None) == _lib.IM2WIN_EINVAL


def test_linear_step_and_backward_refuse():
    L = m.load_library()
    ok = dict(L=1, state_in=FAKE, state_out=FAKE)
    for bad in (dict(L=2), dict(state_in=0), dict(state_out=0), dict(state_out=FAKE + 64), dict(lens=FAKE)):
        assert L.im2win_seq_linear_step(_linear(**{**ok, **bad}), None) == _lib.IM2WIN_EINVAL
    assert L.im2win_seq_linear_step(None, None) == _lib.IM2WIN_EINVAL
    assert L.im2win_seq_linear(None, None, 0, None) == _lib.IM2WIN_EINVAL
    assert L.im2win_seq_linear_backward(None, None, 0, None) == _lib.IM2WIN_EINVAL
    for n in ("dout", "dq", "dk", "dv"):
        for t in BAD_TENSORS:
            assert L.im2win_seq_linear_backward(_linear(**{n: t}), FAKE, 1 << 40, None) == _lib.IM2WIN_EINVAL
    for n in ("dstate_out", "dstate_in"):
        assert L.im2win_seq_linear_backward(_linear(**{n: FAKE + 4}), FAKE, 1 << 40, None) == _lib.IM2WIN_EINVAL


def test_nothing_to_do_is_no_error():
    L = m.load_library()
    none = (0, 0, 0, 0)
    assert L.im2win_seq_attention(_attention(B=0, q=none, k=none, v=none, out=none), None, 0, None) == 0
    assert L.im2win_seq_attention(_attention(Lq=0, q=none, out=none), None, 0, None) == 0
    assert L.im2win_seq_linear(_linear(B=0, q=none, k=none, v=none, out=none), None, 0, None) == 0


# ---- refusals of the binding -------------------------------------------------
def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        m.window_attention(x, x, x, window=2)
    with pytest.raises(ValueError, match="GPU"):
        m.linear_attention(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="GPU"):
        m.linear_attention_step(x[:, 0], x[:, 0], x[:, 0], torch.zeros(2), torch.zeros(1, 2, 64, 64))


def test_workspace_queries():
    # One row of one head over a long cache is split; a full batch of prompts is not.
    assert m.window_attention_workspace_bytes(1, 1, 8192, 8, 1, 128, window=4096) > 0
    assert m.window_attention_workspace_bytes(8, 4096, 4096, 32, 8, 128, window=1024) == 0
    assert m.window_attention_workspace_bytes(1, 300, 300, 4, 2, 64, window=64, backward=True) > 0
    assert m.linear_attention_workspace_bytes(1, 32768, 16, 128, 128) > 0
    assert m.linear_attention_workspace_bytes(1, 16, 16, 128, 128) == 0
