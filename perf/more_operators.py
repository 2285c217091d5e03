"""What stands between the packed products of a decoder layer: the norm with the
residual's addition, the rotation and the paged cache, and the attention that
reads it, each in its plain form and as a user of the library calls it, with the
sizes at which it is measured.

Operators (``case["op"]``):
  norm    x + residual, its root-mean-square norm and the weights
  append  q and k normed (where the model does) and rotated, k and v stored in a paged cache
  causal  attention over the cache: whole prompts, chunks behind a context, single tokens
  tree    the same for drafted tokens that form a tree behind the context
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
K_SCALE, V_SCALE = 0.03125, 0.0625  # of a cache in 8 bits: a calibration's powers of two
EPS = 1e-6
GOLDEN = 0.6180339887498949
LARGEST_SCORES = 40 * 2048 * 2048
LARGEST_BYTES = 1.1e9
LARGEST_FLOPS = 4 * 128 * 40 * 2048 * 2049 // 2


def listed():
    return [
        # one decoded token, hidden size 2048: latency
        dict(name="norm one token", op="norm", M=1, N=2048),
        # a long prompt's rows, hidden size 5120
        dict(name="norm prompt", op="norm", M=4096, N=5120),
        # one decoded token of a small model
        dict(name="append one token", op="append", B=1, n=1, ctx=1000, ragged=False, Hq=32, Hkv=8, D=64, page=16,
             type="f16", norm=False, interleaved=True),
        # packed prompts of a model that norms q and k, into a cache in 8 bits
        dict(name="append prompts", op="append", B=5, n=2048, ctx=0, ragged=True, Hq=32, Hkv=8, D=128, page=64,
             type="e4m3", norm=True, interleaved=False),
        # one decoded token of a small model over a short context: latency
        dict(name="decode one token", op="causal", B=1, n=1, ctx=1000, ragged=False, Hq=32, Hkv=8, D=64, page=16,
             type="f16"),
        # one user's next token behind a long document
        dict(name="decode long context", op="causal", B=1, n=1, ctx=131072, ragged=False, Hq=40, Hkv=8, D=128, page=64,
             type="f16"),
        # a batch of decoding users, contexts of all lengths, a cache in 8 bits
        dict(name="decode batch of 48", op="causal", B=48, n=1, ctx=8192, ragged=True, Hq=32, Hkv=8, D=128, page=32,
             type="e4m3"),
        # the bounded chunk of 32 prompt tokens behind what is in the cache
        dict(name="chunk of 32", op="causal", B=1, n=32, ctx=4000, ragged=False, Hq=32, Hkv=8, D=128, page=64,
             type="bf16"),
        # a whole prompt: the largest product
        dict(name="prompt of 2048", op="causal", B=1, n=2048, ctx=0, ragged=False, Hq=40, Hkv=8, D=128, page=64,
             type="f16"),
        # packed prompts of different lengths
        dict(name="packed prompts", op="causal", B=7, n=1531, ctx=0, ragged=True, Hq=32, Hkv=8, D=64, page=16,
             type="bf16"),
        # one user's drafted tokens
        dict(name="tree of 8", op="tree", B=1, n=8, ctx=2000, ragged=False, Hq=32, Hkv=8, D=128, page=64, type="f16"),
        # drafted tokens of a batch, contexts of all lengths
        dict(name="trees of 40", op="tree", B=16, n=40, ctx=4096, ragged=True, Hq=32, Hkv=8, D=128, page=32,
             type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        op = rng.choice(("norm", "append", "causal", "causal", "causal", "tree"))
        if op == "norm":
            case = dict(op=op, M=_log_int(rng, 1, 4096), N=_log_int(rng, 64, 8192))
        else:
            Hkv = _log_int(rng, 1, 16)
            case = dict(op=op, B=_log_int(rng, 1, 64), n=1, ctx=0, ragged=rng.random() < 0.7,
                        Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=rng.choice((64, 64, 80, 96, 128, 128, 128, 256)),
                        page=rng.choice((16, 32, 64, 128)), type=rng.choice(("f16", "bf16", "e4m3")))
            kind = rng.choice(("prompt", "chunk", "token"))
            if op == "tree":
                case.update(n=_log_int(rng, 2, 64), ctx=_log_int(rng, 1, 20000))
            elif kind == "prompt":
                case.update(n=_log_int(rng, 2, 4096))
            elif kind == "chunk":
                case.update(n=_log_int(rng, 2, 512), ctx=_log_int(rng, 1, 20000))
            else:
                case.update(ctx=_log_int(rng, 1, 131072))
            if op == "append":
                case.update(norm=rng.random() < 0.5, interleaved=rng.random() < 0.5)
            sizes = _sizes(case)
            # the plain form's scores and the keys and values it gathers, in 32 bits, padded to the longest
            longest, most = max(c + n for c, n in sizes), max(n for c, n in sizes)
            if case["B"] * case["Hq"] * most * longest > LARGEST_SCORES:
                continue
            if 8 * case["B"] * case["Hkv"] * longest * case["D"] > 4e9:
                continue
        w = work(case)
        if w["flops"] <= LARGEST_FLOPS and w["bytes"] <= LARGEST_BYTES:
            return case


def _sizes(case):
    """(context, new tokens) of each sequence."""
    out = []
    for b in range(case["B"]):
        part = 1.0 if b == 0 or not case["ragged"] else (b * GOLDEN) % 1.0
        out.append((int(case["ctx"] * part), max(1, int(math.ceil(case["n"] * part)))))
    return out


def work(case):
    if case["op"] == "norm":
        M, N = case["M"], case["N"]
        return {"bytes": 16 * M * N + 4 * N, "flops": 5 * M * N}
    sizes = _sizes(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = sum(n for _, n in sizes)
    size = 1 if case["type"] == "e4m3" else 2
    table = 4 * sum(-(-(c + n) // case["page"]) for c, n in sizes) + 8 * case["B"] + 4
    if case["op"] == "append":
        return {"bytes": T * D * (8 * Hq + 8 * Hkv + 2 * Hkv * size) + table + 2 * D + 8 * D * case["norm"],
                "flops": T * D * (6 * Hq + 6 * Hkv)}
    keys = sum(c + n for c, n in sizes)
    if case["op"] == "tree":
        pairs = sum(n * c + n * max(1, int(math.log2(n + 1))) for c, n in sizes)
        table += 4 * T * _words(case)
    else:
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in sizes)
    return {"bytes": 8 * T * Hq * D + 2 * keys * Hkv * D * size + table, "flops": 4 * D * Hq * pairs}


def _words(case):
    return (case["n"] + 31) // 32


# ---- inputs -----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "norm":
        M, N = case["M"], case["N"]
        # a residual stream: a few channels much larger than the others
        s["residual"] = randn(M, N) * (1.0 + 20.0 * (rand(1, N) < 0.01))
        s["x"], s["weight"] = 0.3 * randn(M, N), 0.5 + rand(N)
        return s
    sizes = _sizes(case)
    B, Hq, Hkv, D, page, dtype = (case[k] for k in ("B", "Hq", "Hkv", "D", "page", "type"))
    dtype = DTYPES[dtype]
    T = sum(n for _, n in sizes)
    need = [-(-(c + n) // page) for c, n in sizes]
    pages = sum(need) + 3
    # the pool's pages lie in any order; the table is padded with -1
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    s["pages"] = table
    s["lengths"] = torch.tensor([c + n for c, n in sizes], dtype=torch.int32, device="cuda")
    s["offsets"] = torch.tensor([0] + [n for _, n in sizes], device="cuda").cumsum(0).int()
    s["k_scale"], s["v_scale"] = (K_SCALE, V_SCALE) if case["type"] == "e4m3" else (1.0, 1.0)
    # keys have a mean that the softmax does not see but the products do
    s["cache_k"] = ((randn(pages, Hkv, page, D) + randn(1, Hkv, 1, D)) / s["k_scale"]).clamp(-448, 448).to(dtype)
    s["cache_v"] = (randn(pages, Hkv, page, D) / s["v_scale"]).clamp(-448, 448).to(dtype)
    s["q"] = 1.5 * randn(T, Hq, D)
    if case["op"] == "append":
        s["k"], s["v"] = 1.5 * randn(T, Hkv, D) + randn(1, Hkv, D), randn(T, Hkv, D)
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
        s["q_norm"], s["k_norm"] = (0.5 + rand(D), 0.5 + rand(D)) if case["norm"] else (None, None)
    if case["op"] == "tree":
        # each drafted token follows an earlier one, or the last token of the context
        words, rows = _words(case), []
        parent = rand(T).tolist()
        for _, n in sizes:
            seen = []
            for i in range(n):
                up = int(parent[len(rows)] * (i + 1)) - 1
                seen.append((seen[up] if up >= 0 else 0) | 1 << i)
                rows.append([seen[i] >> 32 * w & 0xFFFFFFFF for w in range(words)])
        bits = torch.tensor(rows, dtype=torch.int64)
        s["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int().cuda()
    return s


# ---- plain forms --------------------------------------------------------------

def _of_tokens(s):
    """Each token's sequence and its index there."""
    offsets, lengths = s["offsets"].long(), s["lengths"].long()
    t = torch.arange(s["q"].shape[0], device=offsets.device)
    seq = (t[:, None] >= offsets[None, 1:]).sum(1)
    return seq, lengths[seq] - offsets[seq + 1] + t


def _plain_norm(s):
    total = s["x"] + s["residual"]
    return total * torch.rsqrt((total * total).mean(1, keepdim=True) + EPS) * s["weight"], total


def _plain_rotated(s, x, weight, index):
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight
    angle = index.double()[:, None] * s["inv_freq"].double()  # far positions: 32 bits lose the angle
    c, n = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if s["case"]["interleaved"]:
        a, b = x[:, :, 0::2], x[:, :, 1::2]
        return torch.stack((a * c - b * n, b * c + a * n), 3).flatten(2)
    a, b = x.chunk(2, 2)
    return torch.cat((a * c - b * n, b * c + a * n), 2)


def _plain_append(s):
    page, dtype = s["case"]["page"], s["cache_k"].dtype
    seq, index = _of_tokens(s)
    at = s["pages"][seq, index // page].long()
    k = _plain_rotated(s, s["k"], s["k_norm"], index) / s["k_scale"]
    v = s["v"] / s["v_scale"]
    if dtype == torch.float8_e4m3fn:
        k, v = k.clamp(-448, 448), v.clamp(-448, 448)
    raw = torch.uint8 if dtype == torch.float8_e4m3fn else torch.int16
    s["cache_k"].view(raw)[at, :, index % page] = k.to(dtype).view(raw)
    s["cache_v"].view(raw)[at, :, index % page] = v.to(dtype).view(raw)
    return _plain_rotated(s, s["q"], s["q_norm"], index), s["cache_k"], s["cache_v"]


def _plain_attention(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    q, offsets, lengths = s["q"], s["offsets"].long(), s["lengths"].long()
    page, W = case["page"], s["pages"].shape[1]
    T, device = q.shape[0], q.device
    longest, most = min(W * page, case["ctx"] + case["n"]), case["n"]
    key = torch.arange(longest, device=device)
    held = key[None] < lengths[:, None]  # [B, keys]
    at = torch.where(held, s["pages"][:, key // page], 0).long()
    k = s["cache_k"].view(-1, Hkv, page, D)[at, :, (key % page)[None]].float() * s["k_scale"]  # [B, keys, Hkv, D]
    v = s["cache_v"].view(-1, Hkv, page, D)[at, :, (key % page)[None]].float() * s["v_scale"]
    k = k.permute(0, 2, 3, 1).reshape(B * Hkv, D, longest)
    v = torch.where(held[:, :, None, None], v, 0.0).permute(0, 2, 1, 3).reshape(B * Hkv, longest, D)
    # the sequences' queries, padded to the most
    i = torch.arange(most, device=device)
    n = offsets[1:] - offsets[:-1]
    rows = (offsets[:-1, None] + i).clamp(max=T - 1)
    qs = q[rows].view(B, most, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B * Hkv, -1, D)
    z = torch.bmm(qs, k).view(B, Hq, most, longest) / math.sqrt(D)
    before = (lengths - n)[:, None, None]
    if case["op"] == "tree":
        drafted = (key[None, None] - before).expand(B, most, longest)
        words = s["mask"].shape[1]
        bits = s["mask"][rows]  # [B, most, words]
        word = bits.gather(2, (drafted >> 5).clamp(0, words - 1))
        seen = (drafted < 0) | ((drafted < 32 * words) & ((word >> (drafted & 31)) & 1 != 0))
    else:
        seen = key[None, None] <= before + i[None, :, None]
    seen = seen & held[:, None]
    z = z.masked_fill_(~seen[:, None], -torch.inf)
    top = z.max(3, keepdim=True).values
    e = torch.exp(z - torch.where(top == -torch.inf, 0.0, top))
    total = e.sum(3, keepdim=True)
    y = torch.bmm(e.view(B * Hkv, -1, longest), v).view(B, Hq, most, D) / torch.where(total == 0, 1.0, total)
    return y.permute(0, 2, 1, 3)[i[None] < n[:, None]]


def _plain(s):
    op = s["case"]["op"]
    return _plain_norm(s) if op == "norm" else _plain_append(s) if op == "append" else _plain_attention(s)


# ---- one pass -------------------------------------------------------------------

def _own(s):
    import gguf_q4_dequant_amd as q4k
    case = s["case"]
    if case["op"] == "norm":
        return q4k.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
    cache = q4k.KVCache(s["cache_k"], s["cache_v"], s["k_scale"], s["v_scale"])
    seqs = q4k.Sequences(s["offsets"], s["lengths"], s["pages"])
    if case["op"] == "append":
        rotation = q4k.Rotation(s["inv_freq"], case["interleaved"])
        q = q4k.kv_append(s["k"], s["v"], cache, seqs, rotation=rotation, q=s["q"], q_norm=s["q_norm"],
                          k_norm=s["k_norm"], eps=EPS)
        return q, s["cache_k"], s["cache_v"]
    if case["op"] == "tree":
        return q4k.attention_tree(s["q"], cache, seqs, s["mask"])
    return q4k.attention(s["q"], cache, seqs)


def run(state):
    return _own(state) if own else _plain(state)


# ---- from the definitions, in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + s["residual"].double()
        return h / (h.square().sum(1) / case["N"] + EPS).sqrt()[:, None] * s["weight"].double(), h
    page, sizes, D, Hkv = case["page"], _sizes(case), case["D"], case["Hkv"]
    G = case["Hq"] // Hkv
    if case["op"] == "append":
        f = s["inv_freq"].double()

        def turned(x, w, pos):
            x = x.double()
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
            unit = torch.polar(torch.ones_like(f)[None], torch.outer(pos.double(), f))[:, None]
            if case["interleaved"]:
                return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:2], -1, 2)) * unit).flatten(2)
            y = torch.complex(x[..., :D // 2], x[..., D // 2:]) * unit
            return torch.cat((y.real, y.imag), 2)

        ck, cv, q, t = s["cache_k"].double(), s["cache_v"].double(), [], 0
        most = 448.0 if case["type"] == "e4m3" else math.inf
        for b, (c, n) in enumerate(sizes):
            pos = torch.arange(c, c + n, device="cuda")
            at = s["pages"][b].long()[pos // page] * page + pos % page
            for big, new, scale in ((ck, turned(s["k"][t:t + n], s["k_norm"], pos), s["k_scale"]),
                                    (cv, s["v"][t:t + n].double(), s["v_scale"])):
                flat = big.permute(0, 2, 1, 3).reshape(-1, Hkv, D)
                flat[at] = (new / scale).clamp(-most, most)
                big.copy_(flat.view(-1, page, Hkv, D).permute(0, 2, 1, 3))
            q.append(turned(s["q"][t:t + n], s["q_norm"], pos))
            t += n
        return torch.cat(q), ck, cv
    out, t = [], 0
    for b, (c, n) in enumerate(sizes):
        L = c + n
        at = s["pages"][b, :-(-L // page)].long()
        keys = s["cache_k"][at].double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L] * s["k_scale"]
        values = s["cache_v"][at].double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L] * s["v_scale"]
        see = torch.ones(n, L, dtype=torch.bool, device="cuda")
        if case["op"] == "tree":
            m = s["mask"][t:t + n].long() & 0xFFFFFFFF
            for j in range(n):
                see[:, c + j] = (m[:, j // 32] >> (j % 32)) % 2 == 1
        else:
            see = see.tril(c)
        y = torch.empty(n, case["Hq"], D, dtype=torch.float64, device="cuda")
        for h in range(case["Hq"]):
            z = (s["q"][t:t + n, h].double() @ keys[h // G].t().contiguous()) * D ** -0.5
            y[:, h] = torch.softmax(z.masked_fill(~see, -math.inf), 1) @ values[h // G].contiguous()
        out.append(y)
        t += n
    return torch.cat(out)
