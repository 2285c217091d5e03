"""Refusals of the mixture-of-experts and selection entry points: every bad
argument is reported before any device call (no GPU needed)."""
import ctypes
import os

import pytest

import gguf_q4_dequant_amd as q4k

A = 1 << 20  # an aligned, never dereferenced stand-in address


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q4k.LIBRARY_PATH):
        from gguf_q4_dequant_amd import build
        build.build()
    return q4k.library()


def test_route_refusals(lib):
    def call(logits=A, bias=None, M=4, E=8, k=2, flags=0, expert=A, weight=A, offsets=A, rows=A):
        return lib.q4k_moe_route(logits, bias, M, E, k, flags, 1.0, expert, weight, offsets, rows, None)

    for bad in (dict(M=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=100, k=65), dict(flags=4),
                dict(M=2 ** 30, k=2)):
        assert call(**bad) == q4k.ERR_BAD_DIM, bad
    for name in ("logits", "expert", "weight", "offsets", "rows"):
        assert call(**{name: None}) == q4k.ERR_NULL, name
        assert call(**{name: A + 2}) == q4k.ERR_ALIGN, name
    assert call(bias=A + 1) == q4k.ERR_ALIGN
    assert call(M=0, offsets=None) == q4k.ERR_NULL


def test_group_refusals(lib):
    assert lib.q4k_moe_group(A, -1, 4, A, A, None) == q4k.ERR_BAD_DIM
    assert lib.q4k_moe_group(A, 4, 0, A, A, None) == q4k.ERR_BAD_DIM
    assert lib.q4k_moe_group(A, 4, 1025, A, A, None) == q4k.ERR_BAD_DIM
    assert lib.q4k_moe_group(None, 4, 4, A, A, None) == q4k.ERR_NULL
    assert lib.q4k_moe_group(A, 4, 4, None, A, None) == q4k.ERR_NULL
    assert lib.q4k_moe_group(A, 4, 4, A, None, None) == q4k.ERR_NULL
    assert lib.q4k_moe_group(A + 1, 4, 4, A, A, None) == q4k.ERR_ALIGN


def test_grouped_refusals(lib):
    def product(w=A, x=A, x_div=1, offsets=A, rows=A, y=A, E=4, P=8, N=16, K=256):
        return lib.q4k_matmul_grouped(w, x, x_div, offsets, rows, y, E, P, N, K, None)

    def swiglu(w=A, w2=A, x=A, x_div=1, offsets=A, rows=A, y=A, E=4, P=8, N=16, K=256):
        return lib.q4k_matmul_grouped_swiglu(w, w2, x, x_div, offsets, rows, y, E, P, N, K, None)

    for call in (product, swiglu):
        for bad in (dict(E=0), dict(E=1025), dict(P=-1), dict(N=-1), dict(K=-256), dict(K=0), dict(K=300), dict(K=2 ** 26 + 256), dict(x_div=0)):
            assert call(**bad) == q4k.ERR_BAD_DIM, bad
        for name in ("w", "x", "offsets", "y"):
            assert call(**{name: None}) == q4k.ERR_NULL, name
        for name in ("w", "x", "y"):
            assert call(**{name: A + 8}) == q4k.ERR_ALIGN, name
        assert call(offsets=A + 2) == q4k.ERR_ALIGN and call(rows=A + 1) == q4k.ERR_ALIGN
        # empty products are no-ops, also without tensors
        assert call(P=0, w=None, x=None, y=None, offsets=None) == q4k.OK
        assert call(N=0, w=None, x=None, y=None, offsets=None) == q4k.OK
    assert swiglu(w2=None) == q4k.ERR_NULL and swiglu(w2=A + 4) == q4k.ERR_ALIGN


def test_combine_refusals(lib):
    def call(w=A, x=A, expert=A, weight=A, offsets=A, rows=A, out=A, E=4, M=4, k=2, N=16, K=256):
        return lib.q4k_matmul_grouped_combine(w, x, expert, weight, offsets, rows, out, E, M, k, N, K, None)

    for bad in (dict(M=-1), dict(k=0), dict(M=2 ** 30), dict(E=0), dict(N=-1), dict(K=0), dict(K=255)):
        assert call(**bad) == q4k.ERR_BAD_DIM, bad
    for name in ("w", "x", "expert", "weight", "offsets", "rows", "out"):
        assert call(**{name: None}) == q4k.ERR_NULL, name
        assert call(**{name: A + 2}) == q4k.ERR_ALIGN, name
    assert call(M=0, w=None, x=None, out=None) == q4k.OK


def test_selection_refusals(lib):
    def struct(**fields):
        a = q4k._Adjustment()
        for n, v in fields.items():
            setattr(a, n, v)
        return ctypes.byref(a)

    ok = struct()

    def adjust(logits=A, out=A, a=ok, M=2, N=64):
        return lib.q4k_logits_adjust(logits, out, a, M, N, None)

    def choose(logits=A, a=ok, M=2, N=64, index=A, value=A):
        return lib.q4k_logits_argmax(logits, a, M, N, index, value, None)

    def head(w=A, x=A, a=ok, M=2, N=64, K=256, index=A, value=A):
        return lib.q4k_matmul_argmax_adjusted(w, x, a, M, N, K, index, value, None)

    for call in (adjust, choose, head):
        assert call(M=-1) == q4k.ERR_BAD_DIM and call(N=-1) == q4k.ERR_BAD_DIM
        assert call(a=None) == q4k.ERR_NULL
        assert call(a=struct(history_len=-1)) == q4k.ERR_BAD_DIM
        assert call(a=struct(bias_len=-1)) == q4k.ERR_BAD_DIM
        assert call(a=struct(history_len=2 ** 30 + 1, history=A)) == q4k.ERR_BAD_DIM
        assert call(a=struct(bias_len=2 ** 31 - 1, bias_id=A, bias_value=A)) == q4k.ERR_BAD_DIM
        assert call(a=struct(history_len=3)) == q4k.ERR_NULL
        assert call(a=struct(bias_len=3, bias_id=A)) == q4k.ERR_NULL
        for name in ("history", "repetition", "frequency", "presence", "bias_id", "bias_value", "mask"):
            assert call(a=struct(**{name: A + 2})) == q4k.ERR_ALIGN, name
        assert call(M=0) == q4k.OK
    assert adjust(logits=None) == q4k.ERR_NULL and adjust(out=None) == q4k.ERR_NULL
    assert adjust(logits=A + 1) == q4k.ERR_ALIGN and adjust(N=0) == q4k.OK
    assert choose(index=None) == q4k.ERR_NULL and choose(value=A + 1) == q4k.ERR_ALIGN
    assert choose(N=0) == q4k.ERR_BAD_DIM
    assert head(K=0) == q4k.ERR_BAD_DIM and head(K=100) == q4k.ERR_BAD_DIM and head(K=-256) == q4k.ERR_BAD_DIM
    assert head(N=0) == q4k.ERR_BAD_DIM and head(w=None) == q4k.ERR_NULL and head(x=A + 8) == q4k.ERR_ALIGN


def test_binding_refuses_before_any_call():
    import torch
    x, w = torch.zeros((4, 256)), torch.zeros((2, 8, 144), dtype=torch.uint8)
    offsets = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        q4k.matmul_grouped(w, x, offsets)
    with pytest.raises(TypeError):
        q4k.matmul_grouped(w.view(16, 144), x, offsets)
    with pytest.raises(TypeError):
        q4k.matmul_grouped_swiglu(w, w, x.double(), offsets)
    with pytest.raises(ValueError, match="device tensor"):
        q4k.moe_route(torch.zeros((2, 8)), 2)
    with pytest.raises(TypeError):
        q4k.moe_route(torch.zeros((2, 8), dtype=torch.float64), 2)
    with pytest.raises(TypeError):
        q4k.moe_group(torch.zeros(4), 2)
    with pytest.raises(ValueError, match="device tensor"):
        q4k.moe_group(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="device tensor"):
        q4k.logits_adjust(torch.zeros((2, 8)), q4k.Adjustment())
    with pytest.raises(TypeError):
        q4k.logits_argmax(torch.zeros(8), q4k.Adjustment())
    with pytest.raises(ValueError, match="together"):
        q4k.Adjustment(bias_id=offsets)
    with pytest.raises(ValueError, match="history"):
        q4k.Adjustment(presence=torch.zeros(1))
    dev = 0
    for bad in (dict(history=torch.zeros((2, 5), dtype=torch.int64)), dict(mask=torch.zeros((2, 2), dtype=torch.int16))):
        with pytest.raises(TypeError):
            q4k.Adjustment(**bad)._checked(dev, 2, 64)
    for bad in (dict(history=torch.zeros((3, 5), dtype=torch.int32)), dict(mask=torch.zeros((2, 1), dtype=torch.int32)),
                dict(history=torch.zeros((2, 5), dtype=torch.int32))):
        with pytest.raises(ValueError):
            q4k.Adjustment(**bad)._checked(dev, 2, 64)


def test_binding_refuses_sizes_that_the_library_cannot_count():
    """The C functions count in int, and ctypes cuts a longer number to its low 32
    bits: 2^32 + 8 would run as 8.  (Tensors without memory: sizes only.)"""
    import torch
    far = (1 << 32) + 8
    meta = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    w, offsets = meta(2, 8, 144, dtype=torch.uint8), meta(3, dtype=torch.int32)
    rows = meta(far, dtype=torch.int32)
    for call in (lambda: q4k.moe_group(rows, 4),
                 lambda: q4k.moe_route(meta(far, 1), 1),
                 lambda: q4k.logits_adjust(meta(far, 1), q4k.Adjustment()),
                 lambda: q4k.logits_adjust(meta(1, far), q4k.Adjustment()),
                 lambda: q4k.logits_argmax(meta(1, far), q4k.Adjustment()),
                 lambda: q4k.matmul_grouped(w, meta(far, 256), offsets, rows),
                 lambda: q4k.matmul_grouped(w, meta(1, 256), offsets, rows, x_div=far),
                 lambda: q4k.matmul_grouped(w, meta(1, 256), offsets, meta(9, dtype=torch.int32), x_div=(1 << 32) + 1),
                 lambda: q4k.matmul_grouped(w, meta(9, 256), offsets, x_div=1 << 30),
                 lambda: q4k.matmul_grouped_swiglu(w, w, meta(far, 256), offsets, rows),
                 lambda: q4k.matmul_grouped(meta(2, 8, ((1 << 32) // 256 + 1) * 144, dtype=torch.uint8),
                                            meta(9, (1 << 32) + 256), offsets),
                 lambda: q4k.matmul_grouped_combine(w, meta(far, 256), q4k.Routing(
                     meta(far, 1, dtype=torch.int32), meta(far, 1), offsets, rows))):
        with pytest.raises(q4k.Q4KError) as refused:
            call()
        assert refused.value.code == q4k.ERR_BAD_DIM
    for sizes in ((2, far, 16, 256), (2, 8, far, 256), (2, 8, 16, (1 << 32) + 256), ((1 << 32) + 2, 8, 16, 256)):
        with pytest.raises(q4k.Q4KError):
            q4k.grouped_tile(*sizes)
