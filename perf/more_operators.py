"""Workloads of the operators around a model whose queries and keys are normed for
each head and whose key/value cache is held to a size: the norm with the rotary
positions (forward and backward), the attention weight that each cached key has
been given, and eviction by that weight.

Every case is a dict of plain values. `prepare` makes its inputs from a seed,
`run` makes one pass: with `own` true through the library's public calls,
otherwise in elementary torch operations in 32 bits. `exact` states the same
result in 64 bits from the definitions.

Definitions.
  Norm and rotary positions: a head x of d elements becomes x r w with
  r = 1 / sqrt(mean(x^2) + eps) and w the weights of Q or of K, one for each
  element, then its first rot = 2 n elements form pairs, (i, i + n) in the half
  layout and (2i, 2i + 1) in the interleaved one; pair i of a token at position t
  turns by a = t f_i and is multiplied by c. Gradients: with g the output's
  gradient turned back by -a (and times c), dw = sum of g x r over tokens and
  heads, dx = r (g w - x r mean(g w x r)).
  Cache: pages of 64 tokens. K codes e4m3 [pages, Hk, 64, d], V codes e4m3
  [pages, Hk, d, 64], one scale per page and head for K and one for V.
  Weights of the keys, fp32 [pages, Hk, 64]: for key j of a cache head the sum of
  exp(scale q k_j - LSE) over the query heads that read it and the query rows that
  see it, added to what the key had; keys from start_b on have had nothing. Query
  row t of sequence b sits at position len_b - qlen_b + t and sees key j < len_b
  unless (causal and j > position) or LTS_j <= position < LTE_j; rows t >= qlen_b
  do not count.
  Eviction: each cache head of a sequence keeps n = min(len, keep) tokens: the
  first min(sink, n), the last min(recent, n - those) and of the others those of
  the largest weight, the lower position first where weights are equal. They are
  written in their order to the pages of another table, codes rounded to the scale
  of the new page: the smallest 2^k with absmax / 448 <= 2^k over its tokens, never
  below 2^-100. Slots behind the last token of a page hold zeros.
"""
import math

import torch

own = False

PAGE = 64
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def _norm(name, B, Hq, Hk, N, d, rot, dtype, weights="same", interleaved=False, backward=False,
          strided=False, scaling="none", far=0, docs=1):
    return {"name": name, "op": "norm", "B": B, "Hq": Hq, "Hk": Hk, "N": N, "d": d, "rot": rot,
            "dtype": dtype, "weights": weights, "interleaved": interleaved, "backward": backward,
            "strided": strided, "scaling": scaling, "far": far, "docs": docs}


def _weigh(name, B, H, Hk, N, d, length, ragged=False, mask="causal", window=0, prefix=0, Hm=1,
           fresh=False):
    return {"name": name, "op": "weigh", "B": B, "H": H, "Hk": Hk, "N": N, "d": d,
            "length": length, "ragged": ragged, "mask": mask, "window": window, "prefix": prefix,
            "Hm": Hm, "fresh": fresh}


def _evict(name, B, Hk, d, length, keep, sink, recent, ragged):
    return {"name": name, "op": "evict", "B": B, "Hk": Hk, "d": d, "length": length, "keep": keep,
            "sink": sink, "recent": recent, "ragged": ragged}


def listed():
    return [
        # Q and K of the packed-document training step (32 heads, 32768 tokens,
        # positions that start again with each document)
        _norm("norm_documents", 1, 32, 32, 32768, 128, 128, "bf16", docs=10),
        # the gradients of a step of two long sequences, half of each head
        # rotated, interleaved pairs, weights kept in fp32
        _norm("norm_gradient", 2, 32, 8, 16384, 128, 64, "f16", weights="f32", interleaved=True,
              backward=True),
        # one new token of each of 64 running sequences, far into a long
        # context whose frequencies are scaled by parts
        _norm("norm_token", 64, 32, 8, 1, 128, 128, "bf16", strided=True, scaling="parts",
              far=500000),
        # the gradients of a small fp32 run with an odd length, read out of a fused
        # projection
        _norm("norm_odd_f32", 3, 5, 5, 777, 64, 32, "f32", backward=True, strided=True,
              scaling="linear"),
        # one sequence, one token: latency
        _weigh("weigh_single", 1, 32, 8, 1, 128, 1000),
        # a batch of running sequences of uneven length
        _weigh("weigh_batch", 64, 32, 8, 1, 128, 8192, ragged=True),
        # the window of 4096 keys and the prefix of 2048 at 131072 tokens
        _weigh("weigh_window", 8, 8, 8, 1, 128, 131072, mask="window", window=4096, prefix=2048),
        # four drafted tokens a sequence; smaller heads
        _weigh("weigh_draft", 16, 32, 4, 4, 64, 16384, ragged=True),
        # the last 512 tokens of a prompt weigh all of it before it is cut down
        _weigh("weigh_prompt", 2, 32, 8, 512, 128, 32768, ragged=True, fresh=True),
        # a few short sequences, odd numbers: latency
        _evict("evict_odd", 3, 4, 64, 1000, 333, 4, 50, True),
        # a batch of sequences cut down to a quarter
        _evict("evict_batch", 64, 8, 128, 8192, 2048, 4, 256, True),
        # two long contexts cut down to an eighth
        _evict("evict_long", 2, 8, 128, 131072, 16384, 64, 1024, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "weigh", "weigh", "evict"])
    while True:
        d = rng.choice([64, 128])
        if op == "norm":
            Hk = _log(rng, 1, 32)
            d = rng.choice([64, 128, 128, 80, 96, 256])
            dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
            c = _norm("", _log(rng, 1, 64), Hk * rng.choice([1, 1, 2, 4, 5]), Hk,
                      _log(rng, 1, 32768), d, rng.choice([d, d, d // 2, d // 4, d - 10, 0]), dtype,
                      rng.choice(["same", "f32"]), rng.random() < 0.4, rng.random() < 0.5,
                      rng.random() < 0.4, rng.choice(["none", "linear", "parts"]),
                      rng.choice([0, 0, 100000, 1000000]), rng.choice([1, 1, 3]))
            fits = c["B"] * (c["Hq"] + c["Hk"]) * c["N"] * d * (2 if dtype == "f32" else 1) \
                <= 32 * 32768 * 128 * (1 if c["backward"] else 2)
        elif op == "weigh":
            Hk = rng.choice([1, 2, 4, 8, 8, 16])
            H = Hk * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
            N = rng.choice([1, 1, 1, 2, 3, 4, 8, _log(rng, 2, 512), _log(rng, 2, 512)])
            mask = rng.choice(["causal", "causal", "window", "documents", "all"])
            c = _weigh("", _log(rng, 1, 128), H, Hk, N, d, max(N, _log(rng, 1, 131072)),
                       rng.random() < 0.7, mask, _log(rng, 8, 8192), rng.choice([0, 64, 1000]),
                       rng.choice([1, 1, Hk, H]), rng.random() < 0.4)
            keys = c["B"] * c["length"]
            fits = keys * Hk * d <= 8 * 131072 * 8 * 128 and keys * H * N <= 2 * 32768 * 32 * 512 \
                and keys * H * N * d <= 2 * 32768 * 32 * 512 * 128
        else:
            length = _log(rng, 1, 131072)
            c = _evict("", _log(rng, 1, 128), rng.choice([1, 2, 4, 8, 8, 16]), d, length,
                       max(1, int(length * rng.choice([0.05, 0.125, 0.25, 0.5, 0.9, 1.1]))),
                       rng.choice([0, 0, 4, 64]), rng.choice([0, 16, 100, 1000]),
                       rng.random() < 0.7)
            fits = c["B"] * length * c["Hk"] * d <= 64 * 8192 * 8 * 128
        if fits:
            del c["name"]
            return c


def _lengths(case):
    """Cached tokens of each sequence (the new ones among them) and live query rows."""
    B, N, top = case["B"], case.get("N", 1), case["length"]
    lens, live = [], []
    for b in range(B):
        u = (b * 0.6180339887 + 0.35) % 1.0
        lens.append(max(1, int(top * (0.2 + 0.8 * u))) if case["ragged"] and b else top)
        live.append(max(1, N - b % 3) if case["ragged"] else N)
    return lens, [min(n, m) for n, m in zip(live, lens)]


def _keeps(case):
    """Tokens that each sequence may keep."""
    return [max(1, case["keep"] - 7 * (b % 4)) if case["ragged"] else case["keep"]
            for b in range(case["B"])]


def work(case):
    d = case["d"]
    if case["op"] == "norm":
        n = case["B"] * (case["Hq"] + case["Hk"]) * case["N"]
        size = 4 if case["dtype"] == "f32" else 2
        passes = 3 if case["backward"] else 2
        return {"bytes": passes * n * d * size + 4 * case["B"] * case["N"],
                "flops": n * (3 * case["rot"] + (12 if case["backward"] else 4) * d)}
    lens, live = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(n, m) for n, m in zip(lens, _keeps(case))) * case["Hk"]
        return {"bytes": 4 * sum(lens) * case["Hk"] + kept * (4 * d + 8), "flops": 2 * kept * d}
    total_bytes, flops = 0, 0
    for n, q in zip(lens, live):
        keys = n
        if case["mask"] == "window":
            keys = min(n, case["window"] + case["prefix"] + q - 1)
        elif case["mask"] == "documents":
            keys = min(n, (n - 1) % max(case["window"], 1) + q)
        old = 0 if case["fresh"] else keys
        new = n if case["fresh"] else keys
        total_bytes += case["Hk"] * (keys * d + 4 * old + 4 * new) + q * case["H"] * (2 * d + 4)
        flops += 2 * q * case["H"] * d * max(1, keys - (0 if case["mask"] == "all" else q // 2))
    return {"bytes": total_bytes, "flops": flops}


# ---------------------------------------------------------------- inputs
def _frequencies(rot, scaling, base=500000.0, factor=8.0, original=8192):
    """Angle per position of each pair, and the factor on the rotated values."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "parts":
        # pairs that turn often within the original length keep their frequency,
        # slow ones are interpolated, a ramp from 32 turns to 1 between them
        out = []
        for x in f:
            turns = original * x / (2.0 * math.pi)
            g = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            out.append(g * x + (1.0 - g) * x / factor)
        return out, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _table(pages_each, order, at):
    """A page table that takes pages order[at], order[at + 1], .. for each sequence in
    turn. Entries behind a sequence's last page are -1, as a server that maps pages late
    has them."""
    need = torch.tensor(pages_each, device=order.device)
    first = at + torch.cumsum(need, 0) - need
    col = torch.arange(max(pages_each), device=order.device)
    live = col[None, :] < need[:, None]
    idx = torch.where(live, first[:, None] + col[None, :], 0)
    return torch.where(live, order[idx], -1).to(torch.int32).contiguous()


def _order(pages, gen, dev):
    return torch.randperm(pages, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)


def _codes(shape, gen, dev):
    """Normal values as codes, at scales that differ from page to page."""
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for p in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - p),) + tuple(shape[1:]), generator=gen, device=dev)
        codes[p:p + step] = (x * 96.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    k = torch.randint(-8, -5, (shape[0], shape[1]), generator=gen, device=dev)
    return codes, torch.exp2(k.float())


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, d = case["B"], case["d"]
    state = {"case": case, "op": case["op"]}
    randn = lambda shape, dt=torch.bfloat16: torch.randn(shape, generator=gen, device=dev).to(dt)
    if case["op"] == "norm":
        N, Hq, Hk, dt = case["N"], case["Hq"], case["Hk"], DTYPES[case["dtype"]]
        if case["strided"]:  # slices of a fused projection, token-major
            x = randn((B, N, (Hq + 2 * Hk) * d), dt)
            q = x[..., :Hq * d].unflatten(2, (Hq, d)).transpose(1, 2)
            k = x[..., Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d)).transpose(1, 2)
        else:
            q, k = randn((B, Hq, N, d), dt), randn((B, Hk, N, d), dt)
        wt = torch.float32 if case["weights"] == "f32" else dt
        f, c = _frequencies(case["rot"], case["scaling"])
        t = torch.arange(N, device=dev)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=dev)
        span = -(-N // case["docs"])
        state.update(q=q, k=k, freqs=torch.tensor(f, dtype=torch.float64).to(dev), c=c,
                     qw=(1.0 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(wt),
                     kw=(1.0 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(wt),
                     positions=(first + t % span).to(torch.int32).contiguous())
        if case["backward"]:
            state.update(dq=randn((B, Hq, N, d), dt), dk=randn((B, Hk, N, d), dt))
        if own:
            from mask_aware_exact_gb300 import flashmask as fm
            state["ws"] = fm.alloc_norm_workspace(d)
        return state
    Hk = case["Hk"]
    lens, live = _lengths(case)
    pages_each = [-(-n // PAGE) for n in lens]
    pages = sum(pages_each)
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["op"] == "evict":
        keeps = _keeps(case)
        out_each = [-(-min(n, m) // PAGE) for n, m in zip(lens, keeps)]
        order = _order(pages + sum(out_each), gen, dev)
        state["table"] = _table(pages_each, order, 0)
        state["out_table"] = _table(out_each, order, pages)
        pages += sum(out_each)
        state["k8"], state["kscale"] = _codes((pages, Hk, PAGE, d), gen, dev)
        state["v8"], state["vscale"] = _codes((pages, Hk, d, PAGE), gen, dev)
        # heavy tails, and a tenth of the keys that no query has seen
        w = torch.exp(2.0 * torch.randn((pages, Hk, PAGE), generator=gen, device=dev)) / 50.0
        seen = torch.rand((pages, Hk, PAGE), generator=gen, device=dev) > 0.1
        state["weights"] = w * seen
        state["most"] = max(min(n, m) for n, m in zip(lens, keeps))
        state["keep"] = torch.tensor(keeps, dtype=torch.int32, device=dev)
        state["index"] = torch.full((B, Hk, state["most"]), -1, dtype=torch.int32, device=dev)
        if own:
            from mask_aware_exact_gb300 import flashmask as fm
            state["cache"] = fm.KVCache(state["k8"], state["v8"], state["kscale"], state["vscale"])
            state["ws"] = fm.alloc_cache_evict_workspace(B, Hk, state["table"].shape[1])
        return state
    H, N = case["H"], case["N"]
    state["table"] = _table(pages_each, _order(pages, gen, dev), 0)
    state["k8"], state["kscale"] = _codes((pages, Hk, PAGE, d), gen, dev)
    state.update(q=randn((B, H, N, d)), live=torch.tensor(live, dtype=torch.int32, device=dev),
                 lts=None, lte=None, causal=case["mask"] != "all",
                 weights=torch.rand((pages, Hk, PAGE), generator=gen, device=dev) * 0.1,
                 start=torch.zeros(B, dtype=torch.int32, device=dev) if case["fresh"] else None)
    if case["mask"] in ("window", "documents"):
        L, Hm, w = state["table"].shape[1] * PAGE, case["Hm"], case["window"]
        j = torch.arange(L, device=dev, dtype=torch.int32)
        h = torch.arange(Hm, device=dev, dtype=torch.int32)[:, None]
        if case["mask"] == "window":
            lts = torch.where(j[None] < case["prefix"], L, (j[None] + w - h % w).clamp(max=L))
        else:
            lts = ((j[None] // w + 1) * w).clamp(max=L).expand(Hm, L)
        state["lts"] = lts[None].expand(B, Hm, L).to(torch.int32).contiguous()
        state["lte"] = torch.full_like(state["lts"], L)
    state["lse"] = torch.logsumexp(_scores(state), -1)  # as the attention before has left it
    if own:
        from mask_aware_exact_gb300 import flashmask as fm
        # V takes no part; a program has it in its cache
        v8 = torch.zeros((pages, Hk, d, PAGE), dtype=torch.float8_e4m3fn, device=dev)
        state["cache"] = fm.KVCache(state["k8"], v8, state["kscale"], torch.ones_like(state["kscale"]))
        state["mask"] = fm.DeviceMask(state["lts"], state["lte"], None, None, state["causal"])
        state["ws"] = fm.alloc_cache_weights_workspace(B, H, Hk, N, d, state["table"].shape[1])
    return state


# ---------------------------------------------------------------- plain forms
def _turn(x, cos, sin, case):
    """Pairs of the first rot elements turned, in fp32; the others as they are."""
    n, rot = case["rot"] // 2, case["rot"]
    r = x[..., :rot]
    x0, x1 = (r[..., 0::2], r[..., 1::2]) if case["interleaved"] else (r[..., :n], r[..., n:])
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    y = torch.stack((y0, y1), -1).flatten(-2) if case["interleaved"] else torch.cat((y0, y1), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _norm_forward(x, w, cos, sin, case):
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    return _turn(xf * r * w.float(), cos, sin, case).to(x.dtype)


def _norm_backward(dy, x, w, cos, sin, case):
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    xn = xf * r
    g = _turn(dy.float(), cos, -sin, case)
    dw = (g * xn).sum((0, 1, 2))
    g = g * w.float()
    dx = r * (g - xn * (g * xn).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw.to(w.dtype)


def _norm_plain(s):
    case = s["case"]
    a = s["positions"].double()[:, None, :, None] * s["freqs"]
    cos, sin = (torch.cos(a) * s["c"]).float(), (torch.sin(a) * s["c"]).float()
    if not case["backward"]:
        return {"q": _norm_forward(s["q"], s["qw"], cos, sin, case),
                "k": _norm_forward(s["k"], s["kw"], cos, sin, case)}
    dq, dqw = _norm_backward(s["dq"], s["q"], s["qw"], cos, sin, case)
    dk, dkw = _norm_backward(s["dk"], s["k"], s["kw"], cos, sin, case)
    return {"q": dq, "k": dk, "qw": dqw, "kw": dkw}


def _visible(s, keys, rows):
    """[B, Hm or 1, N, L]: which keys each query row sees."""
    pos = (s["lens"] - s["live"])[:, None] + rows
    see = (keys < s["lens"][:, None, None, None]).expand(-1, 1, rows.numel(), -1)
    p = pos[:, None, :, None]
    if s["causal"]:
        see = see & (keys <= p)
    if s["lts"] is not None:
        see = see & ~((s["lts"][:, :, None, :] <= p) & (p < s["lte"][:, :, None, :]))
    return see


def _scores(s):
    """[B, H, N, L]: scores, -inf where a row does not see the key."""
    case = s["case"]
    B, H, Hk, N, d = (case[n] for n in ("B", "H", "Hk", "N", "d"))
    L, t = s["table"].shape[1] * PAGE, s["table"].clamp(min=0).long()
    k = s["k8"].view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * s["kscale"][t][..., None, None]
    k = k.transpose(1, 2).reshape(B, Hk, L, d)
    score = s["q"].float().view(B, Hk, H // Hk * N, d) @ k.transpose(-1, -2)
    del k
    score = score.view(B, H, N, L).mul_(1.0 / math.sqrt(d))
    see = _visible(s, torch.arange(L, device=score.device), torch.arange(N, device=score.device))
    if see.shape[1] > 1:
        see = see.repeat_interleave(H // see.shape[1], 1)
    return score.masked_fill_(~see, -math.inf)


def _weigh_plain(s):
    case = s["case"]
    B, H, Hk, N = (case[n] for n in ("B", "H", "Hk", "N"))
    M = s["table"].shape[1]
    dev = s["q"].device
    rows = (torch.arange(N, device=dev) < s["live"][:, None])[:, None] & (s["lse"] > -math.inf)
    p = _scores(s).sub_(torch.where(rows, s["lse"], math.inf)[..., None]).exp_()
    got = p.view(B, Hk, H // Hk * N, M * PAGE).sum(2).view(B, Hk, M, PAGE).transpose(1, 2)
    j = torch.arange(M * PAGE, device=dev).view(1, M, 1, PAGE)
    start = s["lens"] - s["live"] if s["start"] is None else s["start"]
    old = s["weights"][s["table"].clamp(min=0).long()]
    new = torch.where(j < start[:, None, None, None], old + got, got)
    new = torch.where(j < s["lens"][:, None, None, None], new, old)
    live = s["table"] >= 0
    s["weights"][s["table"][live].long()] = new[live]
    return {"weights": s["weights"]}


def _scale_of(absmax):
    m, e = torch.frexp(absmax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-100)
    k = torch.where(absmax > 0, k, -100)
    return torch.ldexp(torch.ones_like(absmax), k)


def _evict_store(x, codes, scales, pages, live, transposed):
    """Pages x [B, M, Hk, 64, d] of values into the cache."""
    scale = _scale_of(x.abs().amax((-1, -2)))
    c = (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    c = c.transpose(-1, -2) if transposed else c
    codes.view(torch.uint8)[pages] = c[live]
    scales[pages] = scale[live]


def _evict_plain(s):
    case = s["case"]
    B, Hk, d, most = case["B"], case["Hk"], case["d"], s["most"]
    dev, M = s["k8"].device, s["out_table"].shape[1]
    lens = s["lens"].long()[:, None, None]
    n = torch.minimum(lens, s["keep"].long()[:, None, None])
    sink = n.clamp(max=case["sink"])
    recent = (n - sink).clamp(max=case["recent"])
    w = s["weights"][s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2)  # [B, Hk, L]
    j = torch.arange(w.shape[2], device=dev)
    w = torch.where((j < sink) | (j >= lens - recent), math.inf, w)
    w = torch.where(j < lens, w, -math.inf)
    order = torch.argsort(w, dim=-1, descending=True, stable=True)[..., :most]
    r = torch.arange(most, device=dev)
    at = torch.where(r < n, order, 1 << 30).sort(-1).values
    s["index"].copy_(torch.where(r < n, at, s["index"]))
    # the kept tokens, slots of the new pages
    r = torch.arange(M * PAGE, device=dev)
    here = r < n
    at = torch.where(here, torch.nn.functional.pad(at, (0, M * PAGE - most)), 0)
    page = torch.gather(s["table"].clamp(min=0).long()[:, None].expand(B, Hk, -1), 2, at // PAGE)
    hk, slot = torch.arange(Hk, device=dev)[:, None], at % PAGE
    k = s["k8"].view(torch.uint8)[page, hk, slot].view(torch.float8_e4m3fn).float()
    v = s["v8"].view(torch.uint8)[page, hk, :, slot].view(torch.float8_e4m3fn).float()
    k = (k * s["kscale"][page, hk][..., None]).masked_fill_(~here[..., None], 0.0)
    v = (v * s["vscale"][page, hk][..., None]).masked_fill_(~here[..., None], 0.0)
    w = s["weights"][page, hk, slot].masked_fill_(~here, 0.0)
    live = s["out_table"] >= 0
    pages = s["out_table"][live].long()
    _evict_store(k.view(B, Hk, M, PAGE, d).transpose(1, 2), s["k8"], s["kscale"], pages, live, False)
    _evict_store(v.view(B, Hk, M, PAGE, d).transpose(1, 2), s["v8"], s["vscale"], pages, live, True)
    s["weights"][pages] = w.view(B, Hk, M, PAGE).transpose(1, 2)[live]
    return dict({x: s[x] for x in ("k8", "kscale", "v8", "vscale", "weights", "index")},
                lens=n.flatten().to(torch.int32))


def run(state):
    op = state["op"]
    if own:
        from mask_aware_exact_gb300 import flashmask as fm
        case = state["case"]
        if op == "norm":
            how = dict(positions=state["positions"], interleaved=case["interleaved"],
                       mscale=state["c"], eps=EPS)
            if not case["backward"]:
                q, k = fm.flashmask_norm_rope(state["q"], state["k"], state["qw"], state["kw"],
                                              state["freqs"], **how)
                return {"q": q, "k": k}
            dq, dk, dqw, dkw = fm.flashmask_norm_rope_bwd(
                state["dq"], state["dk"], state["q"], state["k"], state["qw"], state["kw"],
                state["freqs"], state["ws"], **how)
            return {"q": dq, "k": dk, "qw": dqw, "kw": dkw}
        if op == "weigh":
            fm.flashmask_cache_weights(state["q"], state["cache"], state["table"], state["lens"],
                                       state["lse"], state["weights"], state["ws"],
                                       mask=state["mask"], q_lens=state["live"],
                                       start=state["start"])
            return {"weights": state["weights"]}
        lens = fm.flashmask_cache_evict(state["cache"], state["table"], state["lens"],
                                        state["weights"], state["keep"], state["ws"],
                                        sink=case["sink"], recent=case["recent"],
                                        out_table=state["out_table"], index=state["index"])
        return dict({x: state[x] for x in ("k8", "kscale", "v8", "vscale", "weights", "index")},
                    lens=lens)
    return {"norm": _norm_plain, "weigh": _weigh_plain, "evict": _evict_plain}[op](state)


# ---------------------------------------------------------------- 64-bit results
def _exact_turn(x, turn, case):
    rot = case["rot"]
    i = torch.arange(rot // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    y = x.clone(memory_format=torch.contiguous_format)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm(s):
    case, out = s["case"], {}
    angle = torch.einsum("bn,i->bni", s["positions"].double(), s["freqs"])
    turn = torch.polar(torch.full_like(angle, s["c"]), -angle if case["backward"] else angle)[:, None]
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "w"].double()
        size = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["d"] + EPS)
        unit = x / size
        if not case["backward"]:
            out[name] = _exact_turn(unit * w, turn, case)
            continue
        g = _exact_turn(s["d" + name].double(), turn, case)
        out[name + "w"] = torch.einsum("bhnd,bhnd->d", g, unit)
        g = g * w
        along = torch.einsum("bhnd,bhnd->bhn", g, unit)[..., None] / case["d"]
        out[name] = (g - unit * along) / size
    return out


def _exact_weigh(s):
    case = s["case"]
    H, Hk, N, d = (case[n] for n in ("H", "Hk", "N", "d"))
    w = s["weights"].double()
    for b, (n, live) in enumerate(zip(s["lens"].tolist(), s["live"].tolist())):
        pages = s["table"][b, :-(-n // PAGE)].long()
        start = n - live if s["start"] is None else int(s["start"][b])
        j = torch.arange(n, device=w.device)
        pos = torch.arange(n - live, n, device=w.device)[:, None]
        for hk in range(Hk):
            k = s["k8"][pages, hk].double() * s["kscale"][pages, hk].double()[:, None, None]
            k = k.reshape(-1, d)[:n]
            mine = w[pages, hk].reshape(-1)
            mine[start:n] = 0.0
            for h in range(hk * (H // Hk), (hk + 1) * (H // Hk)):
                x = s["q"][b, h, :live].double() @ k.T / math.sqrt(d)
                hidden = (j > pos) if s["causal"] else torch.zeros_like(x, dtype=torch.bool)
                if s["lts"] is not None:
                    m = h // (H // s["lts"].shape[1])
                    hidden = hidden | ((s["lts"][b, m, :n] <= pos) & (pos < s["lte"][b, m, :n]))
                p = torch.exp(x - s["lse"][b, h, :live].double()[:, None])
                mine[:n] += torch.where(hidden, 0.0, p).sum(0)
            w[pages, hk] = mine.view(-1, PAGE)
    return {"weights": w}


def _round_e4m3(x):
    """Nearest e4m3 value (ties to even) of 64-bit values of magnitude <= 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _exact_evict(s):
    case = s["case"]
    Hk, d = case["Hk"], case["d"]
    out = {n: s[n].double() for n in ("k8", "kscale", "v8", "vscale", "weights", "index")}
    lens = []
    for b, (n, keep) in enumerate(zip(s["lens"].tolist(), s["keep"].tolist())):
        m = min(n, keep)
        lens.append(m)
        sink = min(case["sink"], m)
        recent = min(case["recent"], m - sink)
        pages, to = s["table"][b].long(), s["out_table"][b].long()
        first, last = torch.arange(sink), torch.arange(n - recent, n)
        for hk in range(Hk):
            w = s["weights"][pages[:-(-n // PAGE)], hk].reshape(-1)[:n].double().cpu()
            middle = torch.sort(w[sink:n - recent], descending=True, stable=True).indices + sink
            kept = torch.cat((first, middle[:m - sink - recent].sort().values, last)).to(pages.device)
            out["index"][b, hk, :m] = kept.double()
            src, slot = pages[kept // PAGE], kept % PAGE
            out["weights"][to[:-(-m // PAGE)], hk] = torch.nn.functional.pad(
                s["weights"][src, hk, slot].double(), (0, -m % PAGE)).view(-1, PAGE)
            for name in ("k", "v"):
                c = s["k8"][src, hk, slot] if name == "k" else s["v8"].view(torch.uint8)[src, hk, :, slot]
                c = c if name == "k" else c.view(torch.float8_e4m3fn)
                x = c.double() * s[name + "scale"][src, hk].double()[:, None]
                x = torch.nn.functional.pad(x, (0, 0, 0, -m % PAGE)).view(-1, PAGE, d)
                top = x.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / 448.0))
                e = e + (top > 448.0 * torch.exp2(e)).double() - (top <= 224.0 * torch.exp2(e)).double()
                scale = torch.exp2(e.clamp(min=-100.0))
                x = _round_e4m3(x / scale[:, None, None])
                out[name + "8"][to[:-(-m // PAGE)], hk] = x if name == "k" else x.transpose(1, 2)
                out[name + "scale"][to[:-(-m // PAGE)], hk] = scale
    out["lens"] = torch.tensor(lens, dtype=torch.int32, device=s["lens"].device)
    out["index"] = out["index"].to(torch.int32)
    return out


def exact(case, seed):
    if case["op"] == "weigh" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "weigh": _exact_weigh, "evict": _exact_evict}[s["op"]](s)
