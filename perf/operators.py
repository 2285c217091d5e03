"""The mixture-of-experts step over packed Q4_K weights, and token selection under
penalties, biases and grammar masks: each operator in its plain form and as a
user of the library calls it, with the sizes at which it is measured.

Operators (``case["op"]``):
  route    router scores -> top-k experts, their weights, and the pairs
           (token, choice) grouped by expert
  grouped  one packed matrix per expert times that expert's rows
  swiglu   the experts' gate and up matrices with silu(g) * u
  combine  the experts' down matrices and the weighted sum over a token's experts
  adjust   penalties, biases and a grammar mask applied to logits
  select   the same, and the greedy choice
"""
import math

import torch

own = False

BLOCK = 256        # weights of a Q4_K super-block
BLOCK_BYTES = 144  # its bytes
LARGEST_FLOPS = 2 * 2048 * 8 * 2 * 1024 * 2048
LARGEST_BYTES = 320e6


def listed():
    return [
        # one decoded token of a model with many small experts: latency
        dict(name="route one token", op="route", M=1, E=128, k=8, sigmoid=False, bias=False),
        # a long prompt under a bias-balanced sigmoid router
        dict(name="route prompt", op="route", M=4096, E=256, k=8, sigmoid=True, bias=True),
        # one token through a plain expert projection, its experts' matrices read once
        dict(name="grouped one token", op="grouped", M=1, E=16, k=2, N=4096, K=2048, skew=0.5),
        # a ragged chunk of a prompt, odd sizes, few large experts
        dict(name="grouped ragged chunk", op="grouped", M=333, E=8, k=2, N=1999, K=1280, skew=1.0),
        # gate and up of one decoded token, many small experts
        dict(name="swiglu one token", op="swiglu", M=1, E=128, k=8, N=1024, K=2048, skew=0.5),
        # a prompt: the largest product
        dict(name="swiglu prompt", op="swiglu", M=2048, E=64, k=8, N=1024, K=2048, skew=0.5),
        # down projections of a batch of decoding users: a few rows for most experts
        dict(name="combine batch of 48", op="combine", M=48, E=64, k=8, N=2048, K=1024, skew=0.5),
        # down projections of a prompt
        dict(name="combine prompt", op="combine", M=1024, E=64, k=8, N=2048, K=1024, skew=0.5),
        # one user's next token under a repetition penalty
        dict(name="select one token", op="select", M=1, N=128256, history=64, bias=0, mask=False),
        # a batch under grammars
        dict(name="select batch under grammars", op="select", M=32, N=151936, history=1024, bias=16, mask=True),
        # a small batch's logits handed to a sampler
        dict(name="adjust batch of 7", op="adjust", M=7, N=32001, history=300, bias=5, mask=True),
        # a large batch's logits handed to a sampler, long histories
        dict(name="adjust batch of 96", op="adjust", M=96, N=128256, history=4096, bias=64, mask=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        op = rng.choice(("route", "grouped", "swiglu", "combine", "adjust", "select"))
        if op == "route":
            E = _log_int(rng, 2, 512)
            case = dict(op=op, M=_log_int(rng, 1, 4096), E=E, k=rng.randint(1, min(E, 16)),
                        sigmoid=rng.random() < 0.5, bias=rng.random() < 0.5)
        elif op in ("grouped", "swiglu", "combine"):
            E = _log_int(rng, 2, 160)
            case = dict(op=op, M=_log_int(rng, 1, 2048), E=E, k=rng.randint(1, min(E, 8)), N=_log_int(rng, 1, 4500),
                        K=BLOCK * _log_int(rng, 1, 20), skew=rng.choice((0.0, 0.5, 1.0, 2.0)))
        else:
            M = _log_int(rng, 1, 128)
            case = dict(op=op, M=M, N=_log_int(rng, 1000, 160000), history=rng.choice((0, _log_int(rng, 1, 4096))),
                        bias=rng.choice((0, _log_int(rng, 1, 64))), mask=rng.random() < 0.6)
            if not (case["history"] or case["bias"] or case["mask"]):
                continue
        w = work(case)
        if op in ("grouped", "swiglu", "combine"):
            # the plain form unpacks every expert in 32 bits: 4 GB at most
            if case["E"] * case["N"] * case["K"] * (2 if op == "swiglu" else 1) > 1 << 29:
                continue
        if w["flops"] <= LARGEST_FLOPS and w["bytes"] <= LARGEST_BYTES:
            return case


def _touched(case):
    """Experts that are expected to have rows."""
    M, E, k = case["M"], case["E"], case["k"]
    return E * (1.0 - (1.0 - k / E) ** M)


def work(case):
    op, M = case["op"], case["M"]
    if op == "route":
        E, P = case["E"], M * case["k"]
        return {"bytes": 4 * M * E + 4 * E * case["bias"] + 12 * P + 4 * (E + 1), "flops": 8 * M * E}
    if op in ("grouped", "swiglu", "combine"):
        E, k, N, K = case["E"], case["k"], case["N"], case["K"]
        P, mats = M * k, 2 if op == "swiglu" else 1
        weights = mats * _touched(case) * N * (K // BLOCK) * BLOCK_BYTES
        x = 4 * K * (P if op == "combine" else M)
        y = 4 * N * (M if op == "combine" else P)
        plan = 4 * (E + 1) + 4 * P + (8 * P if op == "combine" else 0)
        return {"bytes": weights + x + y + plan, "flops": 2 * mats * P * N * K}
    N = case["N"]
    side = 4 * M * case["history"] + 8 * M * case["bias"] + (M * ((N + 31) // 32) * 4 if case["mask"] else 0)
    return {"bytes": 4 * M * N + side + (4 * M * N if op == "adjust" else 8 * M), "flops": 4 * M * N}


# ---- inputs -----------------------------------------------------------------

def _weights(g, E, N, K):
    """Packed Q4_K matrices [E, N, K/256*144] of centred weights, about
    1/sqrt(K) in size: uniform quants, scales and mins, binary16 d and dmin."""
    kb = K // BLOCK
    w = torch.randint(0, 256, (E, N, kb, BLOCK_BYTES), generator=g, device="cuda", dtype=torch.uint8)
    d = (torch.rand((E, N, kb, 1), generator=g, device="cuda") + 0.5) / (200.0 * math.sqrt(K))
    dmin = d * 7.5 * (0.8 + 0.4 * torch.rand((E, N, kb, 1), generator=g, device="cuda"))
    w[..., 0:2] = d.half().view(torch.uint8)
    w[..., 2:4] = dmin.half().view(torch.uint8)
    return w.view(E, N, kb * BLOCK_BYTES)


def _grouping(expert, E):
    """offsets [E + 1] and rows of the pairs of a [M, k] table of experts."""
    flat = expert.reshape(-1)
    rows = torch.sort(flat, stable=True).indices.int()
    counts = torch.bincount(flat.long(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = counts.cumsum(0)
    return offsets, rows, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    randint = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    op, M = case["op"], case["M"]
    s = {"case": case}
    if op == "route":
        E = case["E"]
        s["logits"] = randn(M, E) * 1.5 + 0.5 * randn(1, E)
        s["bias"] = 0.1 * randn(E) if case["bias"] else None
        return s
    if op in ("grouped", "swiglu", "combine"):
        E, k, N, K = case["E"], case["k"], case["N"], case["K"]
        # what a router gives: some experts are liked more than others
        score = randn(M, E) + case["skew"] * randn(1, E)
        top = score.topk(k, dim=1)
        s["expert"] = top.indices.int().contiguous()
        s["weight"] = torch.softmax(top.values, dim=1).contiguous()
        s["offsets"], s["rows"], s["most"] = _grouping(s["expert"], E)
        s["x"] = randn(M * k if op == "combine" else M, K)
        s["w"] = _weights(g, E, N, K)
        if op == "swiglu":
            s["w_up"] = _weights(g, E, N, K)
        return s
    N, L, B = case["N"], case["history"], case["bias"]
    s["logits"] = 3.0 * randn(M, N)
    if L:
        # recent tokens: common ones come again and again; a padded start
        ids = (N * rand(M, L) ** 4).int()
        keep = (1 + (L * rand(M, 1)).int()).clamp(max=L)
        s["history"] = torch.where(torch.arange(L, device="cuda")[None] < keep, ids, -1).int().contiguous()
        # the model tends to say again what it has said
        s["logits"].scatter_add_(1, s["history"].clamp(min=0).long(), 0.5 * rand(M, L))
        s["repetition"] = 1.0 + 0.5 * rand(M)
        s["frequency"] = 0.2 * rand(M)
        s["presence"] = 0.5 * rand(M)
    if B:
        s["bias_id"] = randint(0, N, M, B)
        s["bias_value"] = 4.0 * randn(M, B)
    if case["mask"]:
        # grammars that leave much, little, and (the last row of a batch) nothing
        words = (N + 31) // 32
        bits = randint(0, 1 << 31, M, words) ^ (randint(0, 2, M, words) << 31)
        few = bits & randint(0, 1 << 31, M, words) & randint(0, 1 << 31, M, words) & randint(0, 1 << 31, M, words)
        s["mask"] = torch.where(torch.arange(M, device="cuda")[:, None] % 2 == 0, bits, few).int().contiguous()
        if M >= 4:
            s["mask"][M - 1] = 0
    return s


# ---- plain forms --------------------------------------------------------------

def _unpack(w):
    """The 32-bit weights [..., N, K] of packed matrices [..., N, K/256*144]."""
    b = w.reshape(*w.shape[:-1], -1, BLOCK_BYTES)
    d = b[..., 0:2].contiguous().view(torch.float16).float()
    dmin = b[..., 2:4].contiguous().view(torch.float16).float()
    s = b[..., 4:16]
    scale = torch.cat([s[..., 0:4] & 63, (s[..., 8:12] & 15) | ((s[..., 0:4] >> 6) << 4)], -1)
    least = torch.cat([s[..., 4:8] & 63, (s[..., 8:12] >> 4) | ((s[..., 4:8] >> 6) << 4)], -1)
    q = b[..., 16:].reshape(*b.shape[:-1], 4, 32)
    q = torch.stack([q & 15, q >> 4], -2).reshape(*b.shape[:-1], 8, 32)
    out = (d * scale)[..., None] * q - (dmin * least)[..., None]
    return out.reshape(*w.shape[:-1], -1)


def _plain_products(s, mats, x_div):
    """y[p] = x[p / x_div] . W[expert of p]^T for every pair p, for each of mats."""
    expert, x = s["expert"].reshape(-1).long(), s["x"]
    P, E = expert.numel(), mats[0].shape[0]
    pair = torch.arange(P, device=x.device)
    if P <= E:
        # few pairs: each takes its expert's matrix
        xp = x[pair // x_div][:, :, None]
        return [torch.bmm(_unpack(w[expert]), xp)[:, :, 0] for w in mats]
    # every expert times its rows, padded to the longest group
    offsets, rows = s["offsets"].long(), s["rows"].long()
    at = (offsets[:-1, None] + torch.arange(s["most"], device=x.device)).clamp(max=P - 1)
    xe = x[rows[at] // x_div].transpose(1, 2).contiguous()
    place = torch.empty_like(rows)
    place[rows] = pair
    rank = place - offsets[expert]
    return [torch.bmm(_unpack(w), xe)[expert, :, rank] for w in mats]


def _plain_route(s):
    case, logits, bias = s["case"], s["logits"], s["bias"]
    M, E, k = case["M"], case["E"], case["k"]
    z = logits.double()  # the choice among close scores decides whole numbers
    score = torch.sigmoid(z) if case["sigmoid"] else torch.softmax(z, dim=1)
    by = score if bias is None else score + bias.double()
    expert = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
    weight = score.gather(1, expert)
    weight = (weight / weight.sum(1, keepdim=True)).float()
    flat = expert.reshape(-1)
    rows = torch.sort(flat, stable=True).indices.int()
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    return expert.int(), weight, offsets, rows


def _plain_adjusted(s):
    z, case = s["logits"], s["case"]
    if case["history"]:
        ids = s["history"]
        count = torch.zeros_like(z).scatter_add_(1, ids.clamp(min=0).long(), (ids >= 0).float())
        r = s["repetition"][:, None]
        seen = count > 0
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - s["frequency"][:, None] * count - s["presence"][:, None] * seen
    if case["bias"]:
        z = z + torch.zeros_like(z).scatter_add_(1, s["bias_id"].long(), s["bias_value"])
    if case["mask"]:
        n = torch.arange(case["N"], device=z.device)
        allowed = (s["mask"][:, n >> 5] >> (n & 31)) & 1
        z = torch.where(allowed != 0, z, -torch.inf)
    return z


def _plain(s):
    op = s["case"]["op"]
    if op == "route":
        return _plain_route(s)
    if op == "grouped":
        return _plain_products(s, [s["w"]], s["case"]["k"])[0]
    if op == "swiglu":
        g, u = _plain_products(s, [s["w"], s["w_up"]], s["case"]["k"])
        return g / (1.0 + torch.exp(-g)) * u
    if op == "combine":
        y = _plain_products(s, [s["w"]], 1)[0]
        return (y.view(s["case"]["M"], s["case"]["k"], -1) * s["weight"][:, :, None]).sum(1)
    z = _plain_adjusted(s)
    if op == "adjust":
        return z
    value = z.max(dim=1).values
    n = torch.arange(z.shape[1], device=z.device)
    index = torch.where(z == value[:, None], n, z.shape[1]).min(dim=1).values
    return torch.where(value == -torch.inf, -1, index).int(), value


# ---- one pass -------------------------------------------------------------------

def _adjustment(q4k, s):
    return q4k.Adjustment(history=s.get("history"), repetition=s.get("repetition"), frequency=s.get("frequency"),
                          presence=s.get("presence"), bias_id=s.get("bias_id"), bias_value=s.get("bias_value"),
                          mask=s.get("mask"))


def _own(s):
    import gguf_q4_dequant_amd as q4k
    case = s["case"]
    op = case["op"]
    if op == "route":
        r = q4k.moe_route(s["logits"], case["k"], bias=s["bias"], sigmoid=case["sigmoid"])
        return r.expert, r.weight, r.offsets, r.rows
    if op == "grouped":
        return q4k.matmul_grouped(s["w"], s["x"], s["offsets"], s["rows"], x_div=case["k"])
    if op == "swiglu":
        return q4k.matmul_grouped_swiglu(s["w"], s["w_up"], s["x"], s["offsets"], s["rows"], x_div=case["k"])
    if op == "combine":
        routing = q4k.Routing(s["expert"], s["weight"], s["offsets"], s["rows"])
        return q4k.matmul_grouped_combine(s["w"], s["x"], routing)
    if op == "adjust":
        return q4k.logits_adjust(s["logits"], _adjustment(q4k, s))
    return q4k.logits_argmax(s["logits"], _adjustment(q4k, s))


def run(state):
    return _own(state) if own else _plain(state)


# ---- from the definitions, in 64 bits ---------------------------------------------

def _exact_matrix(w):
    """One packed matrix [N, K/256*144] in 64 bits, sub-block by sub-block."""
    N = w.shape[0]
    b = w.view(-1, BLOCK_BYTES)
    half = lambda at: b[:, at:at + 2].contiguous().view(torch.float16).double()[:, 0]  # noqa: E731
    d, dmin = half(0), half(2)
    t = b[:, 4:16].int()
    out = torch.empty((b.shape[0], 8, 32), dtype=torch.float64, device=w.device)
    for j in range(8):
        if j < 4:
            sc, m = t[:, j] % 64, t[:, j + 4] % 64
        else:
            sc, m = t[:, j + 4] % 16 + 16 * (t[:, j - 4] // 64), t[:, j + 4] // 16 + 16 * (t[:, j] // 64)
        byte = b[:, 16 + 32 * (j // 2):48 + 32 * (j // 2)].int()
        q = byte // 16 if j % 2 else byte % 16
        out[:, j] = (d * sc)[:, None] * q - (dmin * m)[:, None]
    return out.view(N, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "route":
        z = s["logits"].double().cpu()
        if case["sigmoid"]:
            score = 1 / (1 + (-z).exp())
        else:
            e = (z - z.max(1, keepdim=True).values).exp()
            score = e / e.sum(1, keepdim=True)
        by = score if s["bias"] is None else score + s["bias"].double().cpu()
        expert, left = [], by.clone()
        for _ in range(case["k"]):
            best = left.max(1).values
            first = (left == best[:, None]).int().argmax(1)
            expert.append(first)
            left[torch.arange(M), first] = -math.inf
        expert = torch.stack(expert, 1)
        weight = score.gather(1, expert)
        weight = weight / weight.sum(1, keepdim=True)
        groups = [(expert.reshape(-1) == e).nonzero()[:, 0] for e in range(case["E"])]
        offsets = torch.tensor([0] + [len(x) for x in groups]).cumsum(0)
        return expert.int(), weight, offsets.int(), torch.cat(groups).int()
    if op in ("grouped", "swiglu", "combine"):
        k = case["k"]
        P = M * k
        y = torch.zeros((P, case["N"]), dtype=torch.float64, device="cuda")
        off, rows, x = s["offsets"].tolist(), s["rows"].long(), s["x"].double()
        for e in range(case["E"]):
            r = rows[off[e]:off[e + 1]]
            if not len(r):
                continue
            xe = x[r if op == "combine" else r // k]
            ye = xe @ _exact_matrix(s["w"][e]).t().contiguous()
            if op == "swiglu":
                ye = ye * torch.sigmoid(ye) * (xe @ _exact_matrix(s["w_up"][e]).t().contiguous())
            y[r] = ye
        if op == "combine":
            y = torch.einsum("mkn,mk->mn", y.view(M, k, -1).cpu(), s["weight"].double().cpu())
        return y
    N = case["N"]
    z = s["logits"].double().cpu()
    out = []
    for m in range(M):
        v = z[m].clone()
        if case["history"]:
            ids = s["history"][m].cpu()
            ids, n = ids[ids >= 0].long().unique(return_counts=True)
            r, f, p = (float(s[name][m]) for name in ("repetition", "frequency", "presence"))
            v[ids] = torch.where(v[ids] > 0, v[ids] / r, v[ids] * r) - f * n - p
        if case["bias"]:
            for i, b in zip(s["bias_id"][m].tolist(), s["bias_value"][m].double().tolist()):
                v[i] += b
        if case["mask"]:
            word = s["mask"][m].cpu().long() & 0xFFFFFFFF
            bit = (word[:, None] >> torch.arange(32)) & 1
            v[bit.reshape(-1)[:N] == 0] = -math.inf
        out.append(v)
    z = torch.stack(out)
    if op == "adjust":
        return z
    value, index = z.max(1).values, z.argmax(1)
    return torch.where(value == -math.inf, torch.full_like(index, -1), index).int(), value
