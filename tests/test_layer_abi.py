"""Refusals of the norm, cache and attention entry points: every bad argument is
reported before any device call (no GPU needed)."""
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


def cache(**f):
    d = dict(k=A, v=A, type=0, pages=8, kv_heads=2, page_size=16, head_dim=64, k_scale=1.0, v_scale=1.0)
    d.update(f)
    return q4k._Cache(**d)


def seqs(**f):
    d = dict(offsets=A, lengths=A, pages=A, count=2, max_pages=4)
    d.update(f)
    return q4k._Sequences(**d)


def test_norm_refusals(lib):
    def call(x=A, residual=None, weight=A, total=None, y=A, M=2, N=8):
        return lib.q4k_rms_norm(x, residual, weight, 1e-6, total, y, M, N, None)

    assert call(M=-1) == q4k.ERR_BAD_DIM and call(N=-1) == q4k.ERR_BAD_DIM
    assert call(N=(1 << 30) + 1) == q4k.ERR_BAD_DIM
    for name in ("x", "weight", "y"):
        assert call(**{name: None}) == q4k.ERR_NULL, name
    for name in ("x", "residual", "weight", "total", "y"):
        assert call(**{name: A + 2}) == q4k.ERR_ALIGN, name
    assert call(M=0, x=None) == q4k.OK and call(N=0, y=None) == q4k.OK


BAD_CACHE = [dict(type=3), dict(type=-1), dict(pages=-1), dict(kv_heads=0), dict(kv_heads=1025), dict(kv_heads=3),
             dict(page_size=0), dict(page_size=24), dict(page_size=131072), dict(head_dim=0), dict(head_dim=8),
             dict(head_dim=72), dict(head_dim=272), dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("nan")),
             dict(v_scale=float("inf"))]
BAD_SEQUENCES = [dict(count=-1), dict(count=65536), dict(max_pages=-1), dict(max_pages=(1 << 26) + 1)]
CALLS = ["append", "attention", "tree"]


def make(lib, what):
    def append(q=A, k=A, v=A, c=None, s=None, r=None, q_out=A, T=4, q_heads=4):
        return lib.q4k_kv_append(q, k, v, c or cache(), s or seqs(), r, q_out, T, q_heads, None)

    def attention(q=A, c=None, s=None, out=A, T=4, q_heads=4):
        return lib.q4k_attention(q, c or cache(), s or seqs(), 0.1, out, T, q_heads, None)

    def tree(q=A, c=None, s=None, mask=A, words=1, out=A, T=4, q_heads=4):
        return lib.q4k_attention_tree(q, c or cache(), s or seqs(), mask, words, 0.1, out, T, q_heads, None)

    return dict(append=append, attention=attention, tree=tree)[what]


@pytest.mark.parametrize("what", CALLS)
def test_refusals_that_the_calls_over_a_cache_share(lib, what):
    call = make(lib, what)
    for bad in BAD_CACHE:
        assert call(c=cache(**bad)) == q4k.ERR_BAD_DIM, bad
    for bad in BAD_SEQUENCES:
        assert call(s=seqs(**bad)) == q4k.ERR_BAD_DIM, bad
    for bad in (dict(T=-1), dict(q_heads=-4), dict(q_heads=0), dict(q_heads=5), dict(T=1 << 30)):
        assert call(**bad) == q4k.ERR_BAD_DIM, bad
    for name in ("k", "v"):
        assert call(c=cache(**{name: None})) == q4k.ERR_NULL
        assert call(c=cache(**{name: A + 8})) == q4k.ERR_ALIGN
    for name in ("offsets", "lengths", "pages"):
        assert call(s=seqs(**{name: None})) == q4k.ERR_NULL
        assert call(s=seqs(**{name: A + 1})) == q4k.ERR_ALIGN
    # no tokens, or no sequences: nothing to do, also without arrays
    assert call(T=0, q=None) == q4k.OK
    assert call(s=seqs(count=0, offsets=None, lengths=None, pages=None), q=None) == q4k.OK
    # sizes are looked at all the same
    assert call(T=0, c=cache(page_size=3)) == q4k.ERR_BAD_DIM


def test_null_structs(lib):
    c, s = cache(), seqs()
    assert lib.q4k_kv_append(A, A, A, None, s, None, A, 4, 4, None) == q4k.ERR_NULL
    assert lib.q4k_kv_append(A, A, A, c, None, None, A, 4, 4, None) == q4k.ERR_NULL
    assert lib.q4k_attention(A, None, s, 0.1, A, 4, 4, None) == q4k.ERR_NULL
    assert lib.q4k_attention(A, c, None, 0.1, A, 4, 4, None) == q4k.ERR_NULL
    assert lib.q4k_attention_tree(A, None, s, A, 1, 0.1, A, 4, 4, None) == q4k.ERR_NULL
    assert lib.q4k_attention_tree(A, c, None, A, 1, 0.1, A, 4, 4, None) == q4k.ERR_NULL


def test_append_refusals(lib):
    call = make(lib, "append")

    def rot(**f):
        return q4k._Rotation(**{**dict(inv_freq=A, rotary=64, eps=1e-6), **f})

    for bad in (dict(rotary=-8), dict(rotary=12), dict(rotary=72), dict(interleaved=2)):
        assert call(r=rot(**bad)) == q4k.ERR_BAD_DIM, bad
    for name in ("k", "v", "q_out"):
        assert call(**{name: None}) == q4k.ERR_NULL, name
    assert call(q=None) == q4k.ERR_NULL  # with q_out
    for name in ("q", "k", "v", "q_out"):
        assert call(**{name: A + 4}) == q4k.ERR_ALIGN, name
    for name in ("q_norm", "k_norm", "inv_freq", "positions"):
        assert call(r=rot(**{name: A + 2})) == q4k.ERR_ALIGN, name


def test_attention_refusals(lib):
    for what in ("attention", "tree"):
        call = make(lib, what)
        for name in ("q", "out"):
            assert call(**{name: None}) == q4k.ERR_NULL, name
            assert call(**{name: A + 4}) == q4k.ERR_ALIGN, name
    tree = make(lib, "tree")
    assert tree(mask=None) == q4k.ERR_NULL and tree(mask=A + 2) == q4k.ERR_ALIGN
    assert tree(words=0) == q4k.ERR_BAD_DIM and tree(words=-1) == q4k.ERR_BAD_DIM
    assert tree(T=0, mask=None) == q4k.OK


def test_structs_match_the_header():
    """Sizes of the structs as a C compiler lays them out (pointers first, then 4-byte members)."""
    assert ctypes.sizeof(q4k._Cache) == 2 * 8 + 7 * 4 + 4
    assert ctypes.sizeof(q4k._Sequences) == 3 * 8 + 2 * 4
    assert ctypes.sizeof(q4k._Rotation) == 4 * 8 + 3 * 4 + 4


def test_the_binding_refuses_before_any_call():
    import torch
    f = lambda *s: torch.zeros(s)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c = q4k.KVCache(f(4, 2, 16, 64).half(), f(4, 2, 16, 64).half())
    s = q4k.Sequences(i(2), i(1), i(1, 4))
    with pytest.raises(ValueError, match="device tensor"):
        q4k.rms_norm(f(2, 8), f(8))
    with pytest.raises(TypeError, match="float32"):
        q4k.rms_norm(f(2, 8).half(), f(8))
    with pytest.raises(ValueError, match="device tensor"):
        q4k.attention(f(1, 4, 64), c, s)
    with pytest.raises(TypeError, match="float32"):
        q4k.attention(f(1, 4, 64).half(), c, s)
    with pytest.raises(TypeError, match="dimensions"):
        q4k.attention(f(4, 64), c, s)
    with pytest.raises(ValueError, match="mask"):
        q4k.attention_tree(f(1, 4, 64), c, s, None)
    with pytest.raises(ValueError, match="device tensor"):
        q4k.kv_append(f(1, 2, 64), f(1, 2, 64), c, s)


def test_the_binding_checks_the_cache():
    import torch
    half = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    with pytest.raises(TypeError, match="float16"):
        q4k._checked_cache(q4k.KVCache(half.float(), half.float()), 2, 64, -1)
    with pytest.raises(ValueError, match="page_size"):
        q4k._checked_cache(q4k.KVCache(half[0], half[0]), 2, 64, -1)
    with pytest.raises(ValueError, match="heads of 128"):
        q4k._checked_cache(q4k.KVCache(half, half), 2, 128, -1)
    with pytest.raises(ValueError, match="4 heads of 64"):
        q4k._checked_cache(q4k.KVCache(half, half), 4, 64, -1)
    with pytest.raises(ValueError, match="cache.v"):
        q4k._checked_cache(q4k.KVCache(half, half[:2]), 2, 64, -1)
    with pytest.raises(TypeError, match="cache.v"):
        q4k._checked_cache(q4k.KVCache(half, half.bfloat16()), 2, 64, -1)
    with pytest.raises(ValueError, match="max_pages"):
        q4k._checked_sequences(q4k.Sequences(half, half, half), -1)
