"""Cases and plain forms of the cache operators around the decode step.

  rope     new q/k rows get their rotary positions; k, v and the 2-bit key codes go into the cache
  attend   causal attention of a ragged chunk of new tokens over the (paged) cache
  kept     attention weight of the decode step's kept tokens, added to the per-token totals
  chunk    attention weight of a chunk's rows, added to the per-token totals
  evict    the tokens of largest total weight are kept; K, V, codes and totals move together

`run` computes them with elementary torch operations, or, where `own` is set, with the package.
Ragged lengths come from the case alone, so `work` counts exactly what a pass needs; values come from the seed.
"""
import math
import random

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of a 32-head layer: the smallest call, latency alone
        dict(name="rope token", op="rope", B=1, Hq=32, Hkv=32, N=4096, new=1, page=0, rot=128, inter=False,
             scaling="none", factor=1.0, base=10000.0, far=0, codes=True),
        # a decode batch with grouped heads and a paged cache, positions beyond the cache's slots (it was evicted
        # before), interleaved layout over half of the head
        dict(name="rope batch", op="rope", B=8, Hq=32, Hkv=8, N=2048, new=1, page=16, rot=64, inter=True,
             scaling="linear", factor=4.0, base=10000.0, far=1000000, codes=True),
        # a ragged chunk of prompts, frequencies scaled to 128K
        dict(name="rope chunk", op="rope", B=4, Hq=32, Hkv=8, N=4096, new=4096, page=64, rot=128, inter=False,
             scaling="yarn", factor=32.0, base=10000.0, far=0, codes=True),
        # a few tokens per sequence over short contexts, three query heads per kv head, pages that end inside a tile
        dict(name="attend short", op="attend", B=3, Hq=24, Hkv=8, N=720, new=17, page=48, tail=5),
        # dense decode of a grouped-head batch at 16K..32K: bound by reading the cache
        dict(name="attend tokens", op="attend", B=8, Hq=32, Hkv=8, N=32768, new=1, page=64, tail=0),
        # a chunk of a long prompt: 2048 new tokens over 32K
        dict(name="attend chunk", op="attend", B=1, Hq=32, Hkv=8, N=32768, new=2048, page=16, tail=0),
        # a batch of whole prompts, no grouping, contiguous cache
        dict(name="attend prompts", op="attend", B=4, Hq=32, Hkv=32, N=4096, new=4096, page=0, tail=3),
        # the decode step's kept tokens at 128K, budget 1024
        dict(name="kept 128k", op="kept", B=1, Hq=32, Hkv=32, N=131072, new=1, page=0, budget=1024),
        # the last 64 queries of each prompt weigh its tokens
        dict(name="chunk window", op="chunk", B=8, Hq=32, Hkv=8, N=32768, new=64, page=64, tail=0),
        # a short cache with a few tokens too many
        dict(name="evict short", op="evict", B=2, Hkv=8, N=700, keep=512, sink=4, recent=64, page=0, opage=0),
        # a prompt's paged cache cut to a budget right after prefill
        dict(name="evict prompt", op="evict", B=1, Hkv=32, N=32768, keep=1024, sink=4, recent=64, page=16, opage=0),
        # long caches of a grouped-head batch halved
        dict(name="evict half", op="evict", B=4, Hkv=8, N=32768, keep=16384, sink=0, recent=128, page=64, opage=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "attend", "kept", "chunk", "evict", "evict"])
    Hkv, G = rng.choice([(1, 1), (1, 8), (2, 5), (4, 2), (8, 3), (8, 4), (8, 1), (4, 8), (32, 1)])
    B = _log(rng, 1, 8)
    page = rng.choice([0, 0, 1, 16, 16, 24, 64, 64, 256])
    if op == "rope":
        new = _log(rng, 1, 4096 // B)
        N = new + _log(rng, 1, 2000)
        rot = rng.choice([128, 128, 64, 32, 96])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, N=N, new=new, page=page, rot=rot, inter=rng.random() < 0.5,
                    scaling=scaling, factor=rng.choice([2.0, 8.0, 32.0]), base=rng.choice([10000.0, 500000.0]),
                    far=rng.choice([0, 0, 131072, 1000000]), codes=rng.random() < 0.7)
    if op == "evict":
        N = _log(rng, 16, 32768)
        keep = max(1, min(N, int(N * rng.choice([0.05, 0.25, 0.5, 0.9, 1.0]))))
        return dict(op=op, B=B, Hkv=Hkv if B * Hkv <= 64 else 8, N=N, keep=keep, sink=rng.choice([0, 4]),
                    recent=rng.choice([0, 1, 32, 64]), page=page, opage=rng.choice([0, 0, 16, 64]))
    if op == "kept":
        N = _log(rng, 64, 131072 // B)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, N=N, new=1, page=page, budget=min(N, _log(rng, 1, 2048)))
    N = _log(rng, 8, 32768)
    most = (32 * 2048 * 32768) // (B * Hkv * G * N)  # no more score entries than the largest listed case
    new = max(1, min(N, most, _log(rng, 1, 4096 if op == "attend" else 512)))
    while B > 1 and B * Hkv * N > 8 * 8 * 32768:
        B //= 2
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, N=N, new=new, page=page, tail=rng.choice([0, 0, 7]))


def _sizes(case):
    """Per sequence: new tokens and context length (the new tokens included); from the case alone."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B, N, new = case["B"], case["N"], case.get("new", 0)
    n = [new if b == 0 or new < 2 else r.randint(max(1, new // 4), new) for b in range(B)]
    if case["op"] == "rope":
        return n, [r.randint(0, N - x) + x for x in n]
    whole = new == N  # prompts from their first token on
    return n, [x if whole else max(x, N if b == 0 else r.randint(max(1, N // 2), N)) for b, x in enumerate(n)]


def _seen(case):
    """Pairs (new token, cached token it sees), over all sequences."""
    n, lens = _sizes(case)
    return sum(x * (L - x) + x * (x + 1) // 2 for x, L in zip(n, lens))


def work(case):
    op, Hkv = case["op"], case["Hkv"]
    n, lens = _sizes(case)
    T, row = sum(n), 2 * D
    if op == "rope":
        b = T * (2 * case["Hq"] + 4 * Hkv) * row + (T * Hkv * D // 4 if case["codes"] else 0)
        return dict(bytes=b, flops=T * (case["Hq"] + Hkv) * case["rot"] * 3)
    if op == "attend":
        b = sum(lens) * Hkv * 2 * row + 2 * T * case["Hq"] * row + T * case["Hq"] * 4
        return dict(bytes=b, flops=4 * D * _seen(case) * case["Hq"])
    if op == "kept":
        k = sum(min(case["budget"], L) for L in lens) * case["Hq"]
        return dict(bytes=k * (row + 4 + 8) + T * case["Hq"] * row, flops=2 * D * k)
    if op == "chunk":
        b = sum(lens) * Hkv * (row + 8) + T * case["Hq"] * (row + 4)
        return dict(bytes=b, flops=2 * D * _seen(case) * case["Hq"])
    k = sum(min(case["keep"], L) for L in lens) * Hkv
    return dict(bytes=sum(lens) * Hkv * 4 + 2 * k * (2 * row + D // 4 + 4) + 4 * k, flops=sum(lens) * Hkv)


# ------------------------------------------------------------------ inputs
def _frequencies(rot, base, scaling, factor):
    """Angle per position of each pair, 64 bits, and the factor on cos and sin (trained length 4096 for yarn)."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f, m = base ** (-i / rot), 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32))), min(rot // 2 - 1, math.ceil(at(1)))
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        m = 0.1 * math.log(factor) + 1.0
    return f, m


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _cache(case, g, N, page, empty=False):
    """K, V and the block table (None: contiguous) of B sequences of N tokens; K has four outlier channels per head."""
    B, Hkv = case["B"], case["Hkv"]
    if page:
        per = -(-N // page)
        spare = 3
        pages = torch.randperm(B * per + spare, generator=g, device="cuda")[: B * per].to(torch.int32).view(B, per)
        shape = (B * per + spare, Hkv, page, D)
    else:
        pages, shape = None, (B, Hkv, N, D)
    if empty:
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), pages
    gain = torch.ones(Hkv, 1, D, device="cuda")
    gain[:, 0, :: D // 4] = 20.0
    K = (_randn(g, *shape).mul_(gain)).to(torch.bfloat16)
    V = _randn(g, *shape).to(torch.bfloat16)
    return K, V, pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    n, lens = _sizes(case)
    cu = [sum(n[:b]) for b in range(B + 1)]
    s = dict(case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    T, N = cu[-1], case["N"]
    if op == "rope":
        # the projection's output: one row per token, q, k and v heads side by side
        qkv = _randn(g, T, (case["Hq"] + 2 * Hkv) * D).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([case["Hq"] * D, Hkv * D, Hkv * D], 1))
        s["K"], s["V"], s["table"] = _cache(case, g, N, case["page"])
        s["codes"] = torch.randint(0, 256, s["K"].shape[:-1] + (D // 4,), generator=g, device="cuda", dtype=torch.uint8) if case["codes"] else None
        s["before"] = s["lens"] - (s["cu"][1:] - s["cu"][:-1])  # tokens in the cache before
        at = torch.cat([torch.arange(L - x, L) + case["far"] for x, L in zip(n, lens)])
        s["pos"] = at.to(torch.int32).cuda()
        f, m = _frequencies(case["rot"], case["base"], case["scaling"], case["factor"])
        turns = f / (2 * math.pi)  # below half a turn each: 64-bit fractions of a turn
        s["freqs"], s["mscale"] = (turns * 2.0 ** 64).round().to(torch.int64).cuda(), m
        s["out"] = torch.zeros(T, case["Hq"], D, dtype=torch.bfloat16, device="cuda")
    elif op in ("attend", "chunk"):
        pad = case["tail"]  # rows behind the last sequence, as in a padded batch
        s["q"] = _randn(g, T + pad, case["Hq"], D).to(torch.bfloat16)
        s["K"], s["V"], s["table"] = _cache(case, g, N, case["page"])
        if op == "attend":
            s["out"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(T + pad, case["Hq"], device="cuda")
        else:
            s["lse"] = torch.zeros(T + pad, case["Hq"], device="cuda")
            s["lse"][s["cu"][0]: T] = _lse(s)
            s["mass"] = _randn(g, B, Hkv, N).abs_()
    elif op == "kept":
        s["q"] = _randn(g, B, case["Hq"], D).to(torch.bfloat16)
        s["K"], _, s["table"] = _cache(case, g, N, case["page"])
        s["mass"] = _randn(g, B, Hkv, N).abs_()
        # each head's kept tokens in no particular order, -1 behind the last
        k = case["budget"]
        some = torch.rand(B, case["Hq"], N, generator=g, device="cuda")
        some = some.masked_fill_(torch.arange(N, device="cuda") >= s["lens"][:, None, None], -1.0)
        top, idx = some.topk(k, -1)
        s["idx"] = torch.where(top >= 0, idx, -1).to(torch.int32).contiguous()
    else:
        s["K"], s["V"], s["table"] = _cache(case, g, N, case["page"])
        s["codes"] = torch.randint(0, 256, s["K"].shape[:-1] + (D // 4,), generator=g, device="cuda", dtype=torch.uint8)
        # most tokens hold little weight, a few much, one in eight none at all (ties)
        s["mass"] = _randn(g, B, Hkv, N).mul_(2.0).exp_() * (torch.rand(B, Hkv, N, generator=g, device="cuda") > 0.125)
        s["K2"], s["V2"], s["table2"] = _cache(case, g, case["keep"], case["opage"], empty=True)
        s["codes2"] = torch.zeros(s["K2"].shape[:-1] + (D // 4,), dtype=torch.uint8, device="cuda")
        cap = case["keep"] if s["table2"] is None else s["table2"].shape[1] * case["opage"]
        s["mass2"] = torch.ones(B, Hkv, cap, device="cuda")
    if s.get("table") is not None and "mass" in s:  # the totals cover whole pages
        cap = s["table"].shape[1] * case["page"]
        s["mass"] = torch.nn.functional.pad(s["mass"], (0, cap - N)).contiguous()
    if own:
        from compressed_sparse_kv_fp32_b200 import adamas
        rows = s["q"].shape[0] if "q" in s else B
        s["ws"] = adamas.ChunkWorkspace(rows, B, case.get("Hq", Hkv), Hkv)
    return s


# ------------------------------------------------------------------ plain forms
def _view(x, table):
    """A cache as [B, Hkv, tokens, width] (a copy if it is paged)."""
    if table is None:
        return x
    y = x[table.long()]  # [B, pages, Hkv, page, width]
    return y.transpose(1, 2).flatten(2, 3)


def _put(x, table, b, t, rows):
    """rows [n, Hkv, width] into the cache at tokens t of sequences b."""
    if table is None:
        x[b, :, t] = rows
    else:
        P = x.shape[2]
        x[table[b, t // P].long(), :, t % P] = rows


def _padded(s):
    """q as [B, Hkv, new * G, D] in 32 bits, the rows' numbers and which of them exist, which cached tokens each sees."""
    B, Hkv, C = s["B"], s["Hkv"], s["new"]
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(C, device="cuda")
    n = cu[1:] - cu[:-1]
    row, live = cu[:-1, None] + i, i < n[:, None]
    q = s["q"][row.clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(B, C, Hkv, -1, D).transpose(1, 2).flatten(2, 3)
    at = (lens - n)[:, None] + i
    return q, row, live, at


def _scores(s):
    """Scaled scores [B, Hkv, new, G, tokens] of the padded rows, -inf where a row does not see the token."""
    q, row, live, at = _padded(s)
    K = _view(s["K"], s["table"]).float()
    sc = (q @ K.transpose(-1, -2)).mul_(SCALE).unflatten(2, (s["new"], -1))
    hidden = torch.arange(K.shape[2], device="cuda") > at[..., None]
    return sc.masked_fill_(hidden[:, None, :, None], -math.inf), row, live


def _lse(s):
    sc, row, live = _scores(s)
    m = sc.amax(-1, keepdim=True)
    lse = sc.sub_(m).exp_().sum(-1).log_().add_(m[..., 0])
    return lse.permute(0, 2, 1, 3).flatten(2, 3)[live]


def _pair(x, inter, rot):
    if inter:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., : rot // 2], x[..., rot // 2: rot]


def _unpair(a, b, inter):
    return torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)


def _codes(k):
    """2-bit codes of bf16 rows: the butterfly of the Hadamard rotation stage by stage in 32 bits, three thresholds
    by the row's largest magnitude, four codes to a byte."""
    y = k.float()
    for h in (1, 2, 4, 8, 16, 32, 64):
        y = y.unflatten(-1, (D // (2 * h), 2, h))
        a, b = y[..., 0, :], y[..., 1, :]
        y = torch.stack((a + b, a - b), -2).flatten(-3)
    y = y * torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32, device=k.device)
    half = 0.5 * y.abs().amax(-1, keepdim=True)
    c = 3 - (y < -half).int() - (y < 0).int() - (y < half).int()
    c = c.unflatten(-1, (D // 4, 4))
    return (c[..., 0] * 64 + c[..., 1] * 16 + c[..., 2] * 4 + c[..., 3]).to(torch.uint8)


def _plain_rope(s):
    rot, inter = s["rot"], s["inter"]
    # the angle in fractions of a turn: the 64-bit product wraps by whole turns
    turn = (s["pos"].long()[:, None] * s["freqs"]).double() * (2.0 ** -63 * math.pi)
    c = (turn.cos() * s["mscale"]).float()[:, None]
    n = (turn.sin() * s["mscale"]).float()[:, None]

    def turned(x):
        a, b = _pair(x.float(), inter, rot)
        y = _unpair(a * c - b * n, b * c + a * n, inter)
        return torch.cat((y.to(torch.bfloat16), x[..., rot:]), -1)

    s["out"].copy_(turned(s["q"]))
    k = turned(s["k"])
    cu = s["cu"].long()
    tok = torch.arange(k.shape[0], device="cuda")
    b = torch.searchsorted(cu, tok, right=True) - 1
    t = s["before"].long()[b] + tok - cu[b]
    _put(s["K"], s["table"], b, t, k)
    _put(s["V"], s["table"], b, t, s["v"])
    if s["codes"] is not None:
        _put(s["codes"], s["table"], b, t, _codes(k))
    return dict(q=s["out"], K=s["K"], V=s["V"], codes=s["codes"])


def _plain_attend(s):
    sc, row, live = _scores(s)
    m = sc.amax(-1, keepdim=True).clamp_(min=-1e30)
    l = sc.sub_(m).exp_().sum(-1, keepdim=True)
    o = sc.flatten(2, 3) @ _view(s["V"], s["table"]).float()
    o = (o / l.flatten(2, 3)).unflatten(2, (s["new"], -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = (l.log_() + m)[..., 0].permute(0, 2, 1, 3).flatten(2, 3)
    s["out"][row[live]] = o[live].to(torch.bfloat16)
    s["lse"][row[live]] = lse[live]
    return dict(out=s["out"], lse=s["lse"])


def _plain_kept(s):
    K = _view(s["K"], s["table"])
    B, Hq, k = s["idx"].shape
    G = Hq // s["Hkv"]
    at = s["idx"].long().view(B, s["Hkv"], G * k)
    rows = K.gather(2, at.clamp(min=0)[..., None].expand(-1, -1, -1, D)).float().view(B, s["Hkv"], G, k, D)
    sc = (rows * s["q"].float().view(B, s["Hkv"], G, 1, D)).sum(-1) * SCALE
    sc = sc.masked_fill(at.view(sc.shape) < 0, -math.inf)
    e = (sc - sc.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    p = e / e.sum(-1, keepdim=True)
    s["mass"].scatter_add_(2, at.clamp(min=0), p.flatten(2))
    return s["mass"]


def _plain_chunk(s):
    sc, row, live = _scores(s)
    lse = s["lse"][row.clamp(max=s["lse"].shape[0] - 1)].unflatten(2, (s["Hkv"], -1)).transpose(1, 2)
    p = sc.sub_(lse[..., None]).exp_().masked_fill_(~live[:, None, :, None, None], 0.0)
    s["mass"].add_(p.sum((2, 3)))
    return s["mass"]


def _plain_evict(s):
    B, Hkv, N = s["mass"].shape
    lens = s["lens"].long()
    k = lens.clamp(max=s["keep"])
    t = torch.arange(N, device="cuda")
    L = lens[:, None, None]
    mass = s["mass"].masked_fill((t < s["sink"]) | ((t >= L - s["recent"]) & (t < L)), math.inf)
    order = mass.masked_fill(t >= L, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    j = torch.arange(s["keep"], device="cuda")
    kept = order[..., : s["keep"]].masked_fill(j >= k[:, None, None], N).sort(-1).values
    s["mass2"].zero_()
    b, h, j = (kept < N).nonzero(as_tuple=True)
    src = kept[b, h, j]
    s["mass2"][b, h, j] = s["mass"][b, h, src]
    for old, new in (("K", "K2"), ("V", "V2"), ("codes", "codes2")):
        x, y = s[old], s[new]
        if s["table"] is None:
            rows = x[b, h, src]
        else:
            rows = x[s["table"][b, src // s["page"]].long(), h, src % s["page"]]
        if s["table2"] is None:
            y[b, h, j] = rows
        else:
            y[s["table2"][b, j // s["opage"]].long(), h, j % s["opage"]] = rows
    kept = kept.masked_fill(kept == N, -1).to(torch.int32)
    return dict(K=s["K2"], V=s["V2"], codes=s["codes2"], mass=s["mass2"], kept=kept, lens=k.to(torch.int32))


def run(s):
    op = s["op"]
    if own:
        from compressed_sparse_kv_fp32_b200 import adamas
        ws = s["ws"]
        if op == "rope":
            adamas.rope_append(s["q"], s["k"], s["v"], s["cu"], s["before"], s["K"], s["V"], s["freqs"], ws,
                               positions=s["pos"], interleaved=s["inter"], mscale=s["mscale"], codes=s["codes"],
                               block_table=s["table"], out=s["out"])
            return dict(q=s["out"], K=s["K"], V=s["V"], codes=s["codes"])
        if op == "attend":
            adamas.chunk_attend(s["q"], s["K"], s["V"], s["cu"], s["lens"], ws, block_table=s["table"],
                                out=s["out"], lse=s["lse"])
            return dict(out=s["out"], lse=s["lse"])
        if op == "kept":
            return adamas.accumulate_kept(s["q"], s["K"], s["idx"], s["lens"], s["mass"], ws, block_table=s["table"])
        if op == "chunk":
            return adamas.accumulate_chunk(s["q"], s["K"], s["lse"], s["cu"], s["lens"], s["mass"], ws,
                                           block_table=s["table"])
        kept, lens = adamas.evict(s["K"], s["V"], s["mass"], s["lens"], s["keep"], ws, codes=s["codes"],
                                  n_sink=s["sink"], n_recent=s["recent"], block_table=s["table"], K_out=s["K2"],
                                  V_out=s["V2"], codes_out=s["codes2"], mass_out=s["mass2"], table_out=s["table2"])
        return dict(K=s["K2"], V=s["V2"], codes=s["codes2"], mass=s["mass2"], kept=kept, lens=lens)
    return dict(rope=_plain_rope, attend=_plain_attend, kept=_plain_kept, chunk=_plain_chunk, evict=_plain_evict)[op](s)


# ------------------------------------------------------------------ the definitions in 64 bits
def _tokens(x, s, b, h, at, page):
    """Rows `at` (int64) of one sequence and head, from the definition of the layout."""
    if s is None:
        return x[b, h, at]
    return x[s[b].long()[at // page], h, at % page]


def exact(case, seed):
    """One sequence and head at a time, from the operators' definitions."""
    s = prepare(case, seed)
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    n, lens = _sizes(case)
    G = case.get("Hq", Hkv) // Hkv
    dev = "cuda"
    if op == "rope":
        q, K, V = s["q"].double(), s["K"].double(), s["V"].double()
        k, v = s["k"].double(), s["v"].double()
        f, m = _frequencies(case["rot"], case["base"], case["scaling"], case["factor"])
        rot = case["rot"]
        R = torch.zeros(len(s["pos"]), D, D, dtype=torch.float64, device=dev)  # each token's rotation as a matrix
        for i in range(D):
            R[:, i, i] = 1.0
        angle = (s["pos"].double()[:, None] * f.cuda()).remainder(2 * math.pi)
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
            R[:, a, a] = R[:, b, b] = m * angle[:, i].cos()
            R[:, b, a] = m * angle[:, i].sin()
            R[:, a, b] = -R[:, b, a]
        q, k = q @ R.transpose(1, 2), k @ R.transpose(1, 2)
        t0 = 0
        for b in range(B):
            for i in range(n[b]):
                at = lens[b] - n[b] + i
                where = (b, slice(None), at) if s["table"] is None else (int(s["table"][b, at // case["page"]]), slice(None), at % case["page"])
                K[where], V[where] = k[t0 + i], v[t0 + i]
            t0 += n[b]
        return dict(q=q, K=K, V=V, codes=None)
    if op == "kept":
        mass = s["mass"].double()
        for b in range(B):
            for h in range(case["Hq"]):
                at = s["idx"][b, h].long()
                at = at[at >= 0]
                rows = _tokens(s["K"], s["table"], b, h // G, at, case["page"]).double()
                mass[b, h // G, at] += torch.softmax(rows @ s["q"][b, h].double() / math.sqrt(D), 0)
        return mass
    if op == "evict":
        K2, V2, mass2 = s["K2"].double(), s["V2"].double(), s["mass2"].double().zero_()
        kept = torch.full((B, Hkv, case["keep"]), -1, dtype=torch.int32, device=dev)
        for b in range(B):
            L = lens[b]
            k = min(case["keep"], L)
            for h in range(Hkv):
                w = s["mass"][b, h, :L].double()
                first = torch.zeros(L, dtype=torch.bool, device=dev)
                first[: case["sink"]] = True
                first[max(0, L - case["recent"]):] = True
                rank = torch.where(first, w.max() + 1, w)
                floor = rank.topk(k).values[-1]
                sure = rank > floor
                ties = (rank == floor).nonzero()[: k - int(sure.sum()), 0]
                sure[ties] = True
                at = sure.nonzero()[:, 0]
                kept[b, h, :k] = at.to(torch.int32)
                mass2[b, h, :k] = w[at]
                j = torch.arange(k, device=dev)
                for x, y in ((s["K"], K2), (s["V"], V2)):
                    rows = _tokens(x, s["table"], b, h, at, case["page"]).double()
                    if s["table2"] is None:
                        y[b, h, :k] = rows
                    else:
                        y[s["table2"][b].long()[j // case["opage"]], h, j % case["opage"]] = rows
        return dict(K=K2, V=V2, codes=None, mass=mass2, kept=kept, lens=s["lens"].clamp(max=case["keep"]))
    out = s["q"].double() * 0
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=dev)
    mass = s["mass"].double() if op == "chunk" else None
    t0 = 0
    for b in range(B):
        at = torch.arange(lens[b], device=dev)
        mine = torch.arange(lens[b] - n[b], lens[b], device=dev)
        for h in range(Hkv):
            K = _tokens(s["K"], s["table"], b, h, at, case["page"]).double()
            V = _tokens(s["V"], s["table"], b, h, at, case["page"]).double()
            for g in range(h * G, h * G + G):
                sc = s["q"][t0: t0 + n[b], g].double() @ K.T / math.sqrt(D)
                sc.masked_fill_(at > mine[:, None], -math.inf)
                if op == "chunk":
                    mass[b, h, : lens[b]] += (sc - s["lse"][t0: t0 + n[b], g, None].double()).exp().sum(0)
                else:
                    z = torch.logsumexp(sc, 1, keepdim=True)
                    out[t0: t0 + n[b], g] = (sc - z).exp() @ V
                    lse[t0: t0 + n[b], g] = z[:, 0]
        t0 += n[b]
    return mass if op == "chunk" else dict(out=out, lse=lse)
