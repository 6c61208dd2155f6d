"""Sequence operators: window attention with sinks, linear attention with decay.

A binding over the sequence part of libim2win.so (include/im2win_seq.h):

    out = window_attention(q, k, v, window=1024, sinks=4)
    out, lse = window_attention(q, k, v, window=1024, sinks=4, return_lse=True)
    dq, dk, dv = window_attention_backward(dout, q, k, v, out, lse, window=1024, sinks=4)

    out, state = linear_attention(q, k, v, log_decay)              # a prompt
    out = linear_attention_step(q, k, v, log_decay, state)         # a token; state in place
    dq, dk, dv, dstate = linear_attention_backward(dout, q, k, v, log_decay)

Tensors are float16 or bfloat16 on the GPU, (B, tokens, heads, head size) with
any strides that are multiples of 8 elements, the innermost 1; head sizes are
multiples of 8 up to 128. Lengths are int32 tensors on the GPU and are not read
by the host. Calls run on torch's current stream of the tensors' device and do
not synchronise. Gradients are explicit calls; nothing is recorded for autograd.

``ws`` of a call is scratch memory (any GPU tensor of at least the bytes that
the ``*_workspace_bytes`` function names); without it the call takes what it
needs from torch's allocator.
"""
from __future__ import annotations

import functools
import struct

from . import _lib

__all__ = ["window_attention", "window_attention_backward", "window_attention_workspace_bytes",
           "linear_attention", "linear_attention_step", "linear_attention_backward",
           "linear_attention_workspace_bytes"]

# seq_attention and seq_linear of include/im2win_seq.h.
_ATTENTION = struct.Struct("<16q5q11if16q")
_LINEAR = struct.Struct("<16q4q6if4x16q2q")
_NONE = (0, 0, 0, 0)
_NO_GRADS = _NONE * 4
_NO_TAIL = _NO_GRADS + (0, 0)
_torch = _raw_stream = None


def _dtype_code(t):
    global _torch, _raw_stream
    if _torch is None:
        import torch
        # torch.cuda.current_stream(device).cuda_stream without the object in
        # between, which costs as much as the rest of a call's checks.
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch = torch
    dtype = t.dtype
    if dtype is _torch.bfloat16:
        return 1
    if dtype is _torch.float16:
        return 0
    raise TypeError(f"expected float16 or bfloat16 tensors, got {dtype}")


def _tensor(t, name, like, shape):
    """(pointer, batch, token and head stride) of a 16-bit tensor (batch,
    token, head, size), or (batch, head, size) of single tokens."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype is not like.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    if len(shape) == 4:
        sb, sl, sh, sd = t.stride()
        B, L, H, _ = shape
        if L <= 1:
            sl = 0
            if L == 0:
                return _NONE
    else:
        sb, sh, sd = t.stride()
        B, H, _ = shape
        sl = 0
    # The stride of an extent of one means nothing.
    if B <= 1:
        sb = 0
        if B == 0:
            return _NONE
    if H == 1:
        sh = 0
    p = t.data_ptr()
    if sd != 1 or (sb | sl | sh) & 7 or p & 15 or sl >= 1 << 24:
        raise ValueError(f"{name} needs an innermost stride of 1, other strides that are multiples of 8 elements "
                         "(from token to token below 2**24) and a 16-byte aligned start")
    return p, sb, sl, sh


def _output(t, name, like, shape):
    """The output tensor given, or a new one, and its pointer and strides."""
    if t is None:
        t = _torch.empty(shape, dtype=like.dtype, device=like.device)
        if len(shape) == 3:
            return t, (t.data_ptr(), shape[1] * shape[2], 0, shape[2])
        head = shape[2] * shape[3]
        return t, (t.data_ptr(), shape[1] * head, head, shape[3])
    r = _tensor(t, name, like, shape)
    if t.numel() and 0 in [s for s, n in zip(t.stride(), shape) if n > 1]:
        raise ValueError(f"{name} must not overlap itself")
    return t, r


def _ints(t, name, like, shape, contiguous=True):
    if t is None:
        return 0
    if t.dtype is not _torch.int32 or tuple(t.shape) != shape or t.device != like.device:
        raise ValueError(f"{name} must be an int32 tensor of shape {shape} on {like.device}")
    if t.numel() and (not t.is_contiguous() if contiguous else t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _floats(t, name, like, shape):
    if t is None:
        return 0
    if t.dtype is not _torch.float32 or tuple(t.shape) != shape or t.device != like.device:
        raise ValueError(f"{name} must be a float32 tensor of shape {shape} on {like.device}")
    if not t.is_contiguous() or (t.dim() == 4 and t.data_ptr() & 15):
        raise ValueError(f"{name} must be contiguous with a 16-byte aligned start")
    return t.data_ptr()


def _call(name, args, like, ws, need):
    """Runs entry point `name` with `need` bytes of scratch (None: it takes
    none) on like's device."""
    device = like.device
    ptr, size = 0, 0
    if ws is not None:
        if not ws.is_cuda or not ws.is_contiguous() or ws.device != device:
            raise ValueError(f"ws must be a contiguous GPU tensor on {device}")
        if need:
            ptr, size = ws.data_ptr(), ws.numel() * ws.element_size()
    elif need:
        ws = _torch.empty(need, dtype=_torch.uint8, device=device)
        ptr, size = ws.data_ptr(), need
    stream = _raw_stream(device.index)
    args = (args, stream) if need is None else (args, ptr, size, stream)
    fn = getattr(_lib.load(), name)
    if device.index == _torch.cuda.current_device():
        status = fn(*args)
    else:
        with _torch.cuda.device(device):
            status = fn(*args)
    if status:
        _lib.check(status, name)


@functools.lru_cache(maxsize=1024)
def _attention_bytes(B, Lq, Lk, Hq, Hkv, D, window, sinks, backward):
    args = _ATTENTION.pack(*[0] * 21, 0, B, Lq, Lk, Hq, Hkv, D, 0, 0, window, sinks, 1.0, *[0] * 16)
    L = _lib.load()
    return (L.im2win_seq_attention_backward_workspace_bytes if backward
            else L.im2win_seq_attention_workspace_bytes)(args)


@functools.lru_cache(maxsize=1024)
def _linear_bytes(B, L, H, Dk, Dv, backward):
    args = _LINEAR.pack(*[0] * 20, 0, B, L, H, Dk, Dv, 1.0, *[0] * 18)
    lib = _lib.load()
    return (lib.im2win_seq_linear_backward_workspace_bytes if backward else lib.im2win_seq_linear_workspace_bytes)(args)


def _gpu(t, name, dims=4):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    return _dtype_code(t)


def _attention_args(q, k, v, window, sinks, scale, q_lens, kv_lens, page_table):
    """The packed argument up to the outputs, a function of (out, lse, grads),
    the shapes of q and of k and v, and the sizes that scratch memory goes by."""
    code = _gpu(q, "q")
    if k.dim() != 4:
        raise ValueError("k must have 4 dimensions")
    B, Lq, Hq, D = q.shape
    Hkv = k.shape[2]
    page = pages = table = table_stride = 0
    if page_table is None:
        Lk = k.shape[1]
        kv_shape = (B, Lk, Hkv, D)
    else:
        pages, page = k.shape[0], k.shape[1]
        if page_table.dim() != 2:
            raise ValueError("page_table must have 2 dimensions")
        per = page_table.shape[1]
        table = _ints(page_table, "page_table", q, (B, per), contiguous=False)
        table_stride, Lk = page_table.stride(0), per * page
        kv_shape = (pages, page, Hkv, D)
        if page < 1:
            raise ValueError("a page must hold a token")
        if table == 0:  # no pages at all: nothing is there to see
            page = pages = Lk = 0
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads cannot share {Hkv} key heads evenly")
    if D < 8 or D > 128 or D % 8:
        raise ValueError("the head size must be a multiple of 8 from 8 to 128")
    window = max(Lk, 1) if window is None else int(window)
    sinks = int(sinks)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1 and sinks at least 0")
    scale = D ** -0.5 if scale is None else float(scale)
    if scale - scale != 0:
        raise ValueError("scale must be finite")
    tq, tk, tv = _tensor(q, "q", q, (B, Lq, Hq, D)), _tensor(k, "k", q, kv_shape), _tensor(v, "v", q, kv_shape)
    lens = _ints(q_lens, "q_lens", q, (B,)), _ints(kv_lens, "kv_lens", q, (B,))

    window, sinks = min(window, 2**31 - 1), min(sinks, 2**31 - 1)

    def pack(out, lse, grads=_NO_GRADS):
        return _ATTENTION.pack(*tq, *tk, *tv, *out, lse, *lens, table, table_stride, code, B, Lq, Lk, Hq, Hkv, D,
                               page, pages, window, sinks, scale, *grads)

    return pack, (B, Lq, Hq, D), kv_shape, (B, Lq, Lk, Hq, Hkv, D, window, sinks)


def window_attention(q, k, v, *, window=None, sinks=0, scale=None, q_lens=None, kv_lens=None, page_table=None,
                     return_lse=False, out=None, lse=None, ws=None):
    """Causal attention of q (B, Lq, Hq, D) over the last ``window`` keys and
    the first ``sinks`` keys; (B, Lq, Hq, D), or (out, lse) with ``return_lse``,
    lse float32 (B, Hq, Lq).

    k and v are (B, Lk, Hkv, D), Hkv dividing Hq (query head h reads key head
    h // (Hq // Hkv)); with ``page_table`` (int32, (B, pages of a sequence))
    they are pools of pages (pages, page size, Hkv, D), and key j of sequence b
    is in page page_table[b, j // page size].

    Sequence b has kv_lens[b] keys (default Lk, or all the table's pages) and
    q_lens[b] queries (default Lq), its last ones: query i stands at p =
    kv_lens[b] - q_lens[b] + i and sees the keys p - window < j <= p and j <
    min(sinks, p + 1). Without ``window`` every earlier key is seen. ``scale``
    defaults to D ** -0.5. Queries that see nothing, and those past q_lens[b],
    get out 0 and lse -infinity. Keys that no query sees are not read: their
    pages may be gone. A page number outside the pool makes the outputs that
    need it NaN.
    """
    pack, q_shape, _, sizes = _attention_args(q, k, v, window, sinks, scale, q_lens, kv_lens, page_table)
    out, t = _output(out, "out", q, q_shape)
    B, Lq, Hq, _ = q_shape
    p = 0
    if return_lse or lse is not None:
        if lse is None:
            lse = _torch.empty((B, Hq, Lq), dtype=_torch.float32, device=q.device)
        p = _floats(lse, "lse", q, (B, Hq, Lq))
    _call("im2win_seq_attention", pack(t, p), q, ws, _attention_bytes(*sizes, False))
    return (out, lse) if return_lse else out


def window_attention_backward(dout, q, k, v, out, lse, *, window=None, sinks=0, scale=None, q_lens=None,
                              kv_lens=None, dq=None, dk=None, dv=None, ws=None):
    """(dq, dk, dv) of window_attention without pages, from the gradient of its
    output and the ``out`` and ``lse`` that it returned. What lies past a
    sequence's end gets zeros."""
    pack, q_shape, kv_shape, sizes = _attention_args(q, k, v, window, sinks, scale, q_lens, kv_lens, None)
    B, Lq, Hq, _ = q_shape
    tout, tdout = _tensor(out, "out", q, q_shape), _tensor(dout, "dout", q, q_shape)
    if lse is None:
        raise ValueError("lse is needed: call window_attention with return_lse=True")
    p = _floats(lse, "lse", q, (B, Hq, Lq))
    dq, a = _output(dq, "dq", q, q_shape)
    dk, b = _output(dk, "dk", q, kv_shape)
    dv, c = _output(dv, "dv", q, kv_shape)
    _call("im2win_seq_attention_backward", pack(tout, p, (*tdout, *a, *b, *c)), q, ws, _attention_bytes(*sizes, True))
    return dq, dk, dv


def window_attention_workspace_bytes(B, Lq, Lk, Hq, Hkv, D, window=None, sinks=0, backward=False):
    """Scratch bytes of window_attention, or of its backward call, for these
    sizes (Lk: the table's pages times their size for a paged cache)."""
    window = max(Lk, 1) if window is None else int(window)
    return _attention_bytes(B, Lq, Lk, Hq, Hkv, D, window, sinks, bool(backward))


def _linear_sizes(q, k, v, log_decay, scale, dims):
    code = _gpu(q, "q", dims)
    if v.dim() != dims:
        raise ValueError(f"v must have {dims} dimensions")
    H, Dk = q.shape[-2:]
    Dv = v.shape[-1]
    for d in (Dk, Dv):
        if d < 8 or d > 128 or d % 8:
            raise ValueError("head sizes must be multiples of 8 from 8 to 128")
    if H < 1:
        raise ValueError("there must be a head")
    scale = Dk ** -0.5 if scale is None else float(scale)
    if scale - scale != 0:
        raise ValueError("scale must be finite")
    if log_decay is None:
        raise ValueError("log_decay is needed")
    return code, H, Dk, Dv, scale, _floats(log_decay, "log_decay", q, (H,))


def linear_attention(q, k, v, log_decay, *, state=None, scale=None, lens=None, out=None, state_out=None, ws=None):
    """Linear attention with a decay for each head over q, k (B, L, H, Dk) and
    v (B, L, H, Dv): with a = exp(log_decay[h]),

        S_t = a S_(t-1) + k_t v_t^T,    out_t = scale * q_t S_t.

    Returns (out, state): out (B, L, H, Dv), and the state after each
    sequence's last token, float32 (B, H, Dk, Dv). ``state`` is the one before
    the first token (default zeros); ``state_out`` may be ``state`` itself.
    log_decay is float32 (H,), at most 0. ``lens`` (int32, (B,)) are the
    sequences' lengths, default L; out is 0 past them. ``scale`` defaults to
    Dk ** -0.5.
    """
    code, H, Dk, Dv, scale, decay = _linear_sizes(q, k, v, log_decay, scale, 4)
    B, L = q.shape[:2]
    qk, vo, st = (B, L, H, Dk), (B, L, H, Dv), (B, H, Dk, Dv)
    out, t = _output(out, "out", q, vo)
    if state_out is None:
        state_out = _torch.empty(st, dtype=_torch.float32, device=q.device)
    args = _LINEAR.pack(*_tensor(q, "q", q, qk), *_tensor(k, "k", q, qk), *_tensor(v, "v", q, vo), *t, decay,
                        _floats(state, "state", q, st), _floats(state_out, "state_out", q, st),
                        _ints(lens, "lens", q, (B,)), code, B, L, H, Dk, Dv, scale, *_NO_TAIL)
    _call("im2win_seq_linear", args, q, ws, _linear_bytes(B, L, H, Dk, Dv, False))
    return out, state_out


def linear_attention_step(q, k, v, log_decay, state, *, scale=None, out=None):
    """One token of linear_attention: q, k (B, H, Dk), v (B, H, Dv); out (B, H,
    Dv). ``state``, float32 (B, H, Dk, Dv), is updated in place."""
    code, H, Dk, Dv, scale, decay = _linear_sizes(q, k, v, log_decay, scale, 3)
    B = q.shape[0]
    if state is None:
        raise ValueError("state is needed")
    qk, vo = (B, H, Dk), (B, H, Dv)
    out, t = _output(out, "out", q, vo)
    s = _floats(state, "state", q, (B, H, Dk, Dv))
    args = _LINEAR.pack(*_tensor(q, "q", q, qk), *_tensor(k, "k", q, qk), *_tensor(v, "v", q, vo), *t, decay, s, s, 0,
                        code, B, 1, H, Dk, Dv, scale, *_NO_TAIL)
    _call("im2win_seq_linear_step", args, q, None, None)
    return out


def linear_attention_backward(dout, q, k, v, log_decay, *, state=None, dstate=None, scale=None, lens=None,
                              dq=None, dk=None, dv=None, ws=None):
    """(dq, dk, dv, dstate_in) of linear_attention. ``state`` is the one that
    the forward call began with, ``dstate`` the gradient of the one that it
    returned; dstate_in, the gradient of ``state``, is None without one.
    log_decay is a constant of the model and gets no gradient. What lies past a
    sequence's end gets zeros."""
    code, H, Dk, Dv, scale, decay = _linear_sizes(q, k, v, log_decay, scale, 4)
    B, L = q.shape[:2]
    qk, vo, st = (B, L, H, Dk), (B, L, H, Dv), (B, H, Dk, Dv)
    tq, tk, tv = _tensor(q, "q", q, qk), _tensor(k, "k", q, qk), _tensor(v, "v", q, vo)
    tdout = _tensor(dout, "dout", q, vo)
    dq, a = _output(dq, "dq", q, qk)
    dk, b = _output(dk, "dk", q, qk)
    dv, c = _output(dv, "dv", q, vo)
    dstate_in = None
    if state is not None:
        dstate_in = _torch.empty(st, dtype=_torch.float32, device=q.device)
    args = _LINEAR.pack(*tq, *tk, *tv, *_NONE, decay, _floats(state, "state", q, st), 0, _ints(lens, "lens", q, (B,)),
                        code, B, L, H, Dk, Dv, scale, *tdout, *a, *b, *c, _floats(dstate, "dstate", q, st),
                        _floats(dstate_in, "dstate_in", q, st))
    _call("im2win_seq_linear_backward", args, q, ws, _linear_bytes(B, L, H, Dk, Dv, True))
    return dq, dk, dv, dstate_in


def linear_attention_workspace_bytes(B, L, H, Dk, Dv, backward=False):
    """Scratch bytes of linear_attention, or of its backward call."""
    return _linear_bytes(B, L, H, Dk, Dv, bool(backward))
