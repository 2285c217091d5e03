"""Outputs that overlap what a call reads are refused before anything runs (workgroups read other rows
than they write, so such a call would be a race)."""
import pytest

import gguf_q4_dequant_amd as q4k

pytestmark = pytest.mark.gpu


def z(*s):
    import torch
    return torch.zeros(s, device="cuda")


def i(*s):
    import torch
    return torch.zeros(s, dtype=torch.int32, device="cuda")


def layer():
    import torch
    pool = torch.zeros(2, 2, 2, 16, 64, dtype=torch.float16, device="cuda")
    return q4k.KVCache(pool[0], pool[1]), q4k.Sequences(i(2), i(1), i(1, 2)), pool


@pytest.mark.parametrize("call", ["attention", "tree"])
def test_attention(call):
    import torch
    cache, seqs, pool = layer()
    both = z(2, 3, 4, 64)
    mask = both[1].view(torch.int32).view(-1)[:3].view(3, 1)
    run = q4k.attention if call == "attention" else lambda q, c, s, out=None: q4k.attention_tree(q, c, s, i(3, 1), out=out)
    q = both[0]
    run(q, cache, seqs, out=both[1])  # beside it
    with pytest.raises(ValueError, match="out must not overlap q"):
        run(q, cache, seqs, out=q)
    with pytest.raises(ValueError, match="out must not overlap q"):
        run(q, cache, seqs, out=both.view(-1)[256:256 + 768].view(3, 4, 64))
    flat = pool.view(torch.float32).view(-1)
    with pytest.raises(ValueError, match="out must not overlap cache.k"):
        run(q, cache, seqs, out=flat[:768].view(3, 4, 64))
    with pytest.raises(ValueError, match="out must not overlap cache.v"):
        run(q, cache, seqs, out=flat[-768:].view(3, 4, 64))
    if call == "tree":
        with pytest.raises(ValueError, match="out must not overlap mask"):
            q4k.attention_tree(q, cache, seqs, mask, out=both[1])


def test_append():
    import torch
    cache, seqs, pool = layer()
    k, v, both = z(3, 2, 64), z(3, 2, 64), z(2, 3, 4, 64)
    q = both[0]
    q4k.kv_append(k, v, cache, seqs, q=q, q_out=both[1])
    q4k.kv_append(k, v, cache, seqs, q=q, q_out=q)
    with pytest.raises(ValueError, match="q_out must not overlap q"):
        q4k.kv_append(k, v, cache, seqs, q=q, q_out=both.view(-1)[256:256 + 768].view(3, 4, 64))
    few = z(3, 2, 64)
    for name, args in (("k", (few, v)), ("v", (k, few))):
        with pytest.raises(ValueError, match=f"q_out must not overlap {name}"):
            q4k.kv_append(*args, cache, seqs, q=z(3, 2, 64), q_out=few)
    with pytest.raises(ValueError, match="q_out must not overlap cache.k"):
        q4k.kv_append(k, v, cache, seqs, q=q, q_out=pool.view(torch.float32).view(-1)[:768].view(3, 4, 64))


def test_norm():
    import torch
    flat = torch.randn(64 + 12 * 8, device="cuda")
    x, shifted = flat[:64].view(8, 8), flat[8:72].view(8, 8)
    other, w = torch.randn(8, 8, device="cuda"), torch.rand(8, device="cuda")
    for bad in (dict(out=shifted), dict(residual=other, out=shifted), dict(residual=other, total=shifted)):
        with pytest.raises(ValueError, match="must not overlap x"):
            q4k.rms_norm(x, w, **bad)
    with pytest.raises(ValueError, match="must not overlap residual"):
        q4k.rms_norm(other, w, residual=x, total=shifted)
    with pytest.raises(ValueError, match="out must not overlap residual"):
        q4k.rms_norm(x, w, residual=shifted, out=x)  # in place of x, which the residual overlaps
    with pytest.raises(ValueError, match="must not overlap weight"):
        q4k.rms_norm(x, other[3], out=other)
    with pytest.raises(ValueError, match="two tensors"):
        q4k.rms_norm(x, w, residual=x, total=other, out=other.view(8, 8))
    with pytest.raises(ValueError, match="total must not overlap out"):
        big = torch.empty(9, 8, device="cuda")
        q4k.rms_norm(x, w, residual=other, total=big[:8], out=big[1:])
    # what is allowed: each output one of the inputs, or beside them
    want = q4k.rms_norm(x, w, residual=other)
    a, b = x.clone(), other.clone()
    got = q4k.rms_norm(a, w, residual=b, total=b, out=a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a = x.clone()
    assert torch.equal(q4k.rms_norm(a, w, residual=a, out=a)[1], 2 * x)
