"""Workloads of the operators around an 8-bit paged key/value cache: rotary
positions (forward and backward), writing new tokens into the cache, and
attention over it under a column-wise mask.

Every case is a dict of plain values. `prepare` makes its inputs from a seed,
`run` makes one pass: with `own` true through the library's public calls,
otherwise in elementary torch operations in 32 bits. `exact` states the same
result in 64 bits from the definitions.

Definitions.
  Rotary positions: the first rot = 2 n elements of each head form n pairs,
  (i, i + n) in the half layout and (2i, 2i + 1) in the interleaved one. Pair i
  of a token at position t turns by the angle a = t f_i and is multiplied by c:
  (x, y) -> c (x cos a - y sin a, y cos a + x sin a). The gradient is the same
  with -a. The other d - rot elements are copied.
  Cache: pages of 64 tokens. K codes e4m3 [pages, Hk, 64, d], V codes e4m3
  [pages, Hk, d, 64], one scale per page and head for K and one for V, a power
  of two: the smallest 2^k with absmax / 448 <= 2^k over the page's tokens,
  never below 2^-100. A scale only grows while a page fills; the codes already
  there are then rounded again to the larger scale.
  Attention: query row t of sequence b sits at position len_b - qlen_b + t and
  sees key j < len_b unless (causal and j > position) or LTS_j <= position <
  LTE_j. O = softmax(scale q k) v over the visible keys and LSE its log-sum; a
  row that sees nothing gives O = 0, LSE = -inf; rows t >= qlen_b are left as
  they were.
"""
import math

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def _rope(name, B, Hq, Hk, N, d, rot, dtype, interleaved=False, backward=False, strided=False,
          scaling="none", far=0, docs=1):
    return {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hk": Hk, "N": N, "d": d, "rot": rot,
            "dtype": dtype, "interleaved": interleaved, "backward": backward, "strided": strided,
            "scaling": scaling, "far": far, "docs": docs}


def _append(name, B, Hk, N, d, held, ragged):
    return {"name": name, "op": "append", "B": B, "Hk": Hk, "N": N, "d": d, "held": held,
            "ragged": ragged}


def _attend(name, B, H, Hk, N, d, length, ragged=False, mask="causal", window=0, prefix=0, Hm=1):
    return {"name": name, "op": "attend", "B": B, "H": H, "Hk": Hk, "N": N, "d": d,
            "length": length, "ragged": ragged, "mask": mask, "window": window, "prefix": prefix,
            "Hm": Hm}


def listed():
    return [
        # Q and K of the packed-document training step (32 heads, 32768 tokens,
        # positions that start again with each document)
        _rope("rope_documents", 1, 32, 32, 32768, 128, 128, "bf16", docs=10),
        # the gradients of a step of two long sequences, half of each head
        # rotated, interleaved pairs
        _rope("rope_gradient", 2, 32, 8, 16384, 128, 64, "f16", interleaved=True, backward=True),
        # one new token of each of 64 running sequences, far into a long
        # context whose frequencies are scaled by parts
        _rope("rope_token", 64, 32, 8, 1, 128, 128, "bf16", strided=True, scaling="parts",
              far=500000),
        # a small fp32 run with an odd length, read out of a fused projection
        _rope("rope_odd_f32", 3, 5, 5, 777, 64, 32, "f32", strided=True, scaling="linear"),
        # the token that each of 64 running sequences has just produced
        _append("append_token", 64, 8, 1, 128, 4000, True),
        # prompts of uneven length, behind what their sequences hold already
        _append("append_prompts", 4, 8, 8192, 128, 500, True),
        # one sequence, one token: latency
        _attend("attend_single", 1, 32, 8, 1, 128, 1000),
        # a batch of running sequences of uneven length
        _attend("attend_batch", 64, 32, 8, 1, 128, 8192, ragged=True),
        # long contexts
        _attend("attend_long", 8, 32, 8, 1, 128, 131072),
        # the window of 4096 keys and the prefix of 2048 at 131072 tokens
        _attend("attend_window", 8, 8, 8, 1, 128, 131072, mask="window", window=4096, prefix=2048),
        # four drafted tokens a sequence, checked at once; smaller heads
        _attend("attend_draft", 16, 32, 4, 4, 64, 16384, ragged=True),
        # a chunk of a prompt behind what is cached
        _attend("attend_chunk", 2, 32, 8, 512, 128, 32768, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    while True:
        d = rng.choice([64, 128])
        if op == "rope":
            Hk = _log(rng, 1, 32)
            c = _rope("", _log(rng, 1, 64), Hk * rng.choice([1, 1, 2, 4, 5]), Hk,
                      _log(rng, 1, 32768), d, rng.choice([d, d, d // 2, d // 4, d - 10]),
                      rng.choice(["bf16", "bf16", "f16", "f32"]), rng.random() < 0.4,
                      rng.random() < 0.4, rng.random() < 0.4,
                      rng.choice(["none", "linear", "parts"]), rng.choice([0, 0, 100000, 1000000]),
                      rng.choice([1, 1, 3]))
            fits = c["B"] * (c["Hq"] + c["Hk"]) * c["N"] * d * (2 if c["dtype"] == "f32" else 1) \
                <= 2 * 32 * 32768 * 128
        elif op == "append":
            c = _append("", _log(rng, 1, 256), _log(rng, 1, 32), _log(rng, 1, 8192), d,
                        rng.choice([0, _log(rng, 1, 10000)]), rng.random() < 0.7)
            fits = c["B"] * c["Hk"] * c["N"] * d <= 4 * 8 * 8192 * 128 \
                and c["B"] * c["Hk"] * (c["N"] + c["held"] + 64) * d <= 1 << 30
        else:
            Hk = rng.choice([1, 2, 4, 8, 8, 16])
            H = Hk * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
            N = rng.choice([1, 1, 1, 2, 3, 4, 8, _log(rng, 2, 512)])
            mask = rng.choice(["causal", "causal", "window", "documents", "all"])
            c = _attend("", _log(rng, 1, 128), H, Hk, N, d, max(N, _log(rng, 1, 131072)),
                        rng.random() < 0.7, mask, _log(rng, 8, 8192), rng.choice([0, 64, 1000]),
                        rng.choice([1, 1, Hk, H]))
            keys = c["B"] * c["length"]
            fits = keys * Hk * d <= 8 * 131072 * 8 * 128 and keys * H * N <= 2 * 32768 * 32 * 512 \
                and keys * H * N * d <= 2 * 32768 * 32 * 512 * 128
        if fits:
            del c["name"]
            return c


def _lengths(case):
    """Cached tokens of each sequence (the new ones among them) and live query rows."""
    B, N, top = case["B"], case["N"], case["length"]
    lens, live = [], []
    for b in range(B):
        u = (b * 0.6180339887 + 0.35) % 1.0
        lens.append(max(1, int(top * (0.2 + 0.8 * u))) if case["ragged"] and b else top)
        live.append(max(1, N - b % 3) if case["ragged"] else N)
    return lens, [min(n, m) for n, m in zip(live, lens)]


def _held(case):
    """Tokens each sequence holds before new ones are written, and how many are."""
    held, new = [], []
    for b in range(case["B"]):
        u = (b * 0.6180339887 + 0.35) % 1.0
        held.append(int(case["held"] * (0.5 + u)) if case["ragged"] else case["held"])
        new.append(max(1, int(case["N"] * (0.5 + 0.5 * u))) if case["ragged"] and b else case["N"])
    return held, new


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["B"] * (case["Hq"] + case["Hk"]) * case["N"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * d * size + 4 * case["B"] * case["N"], "flops": 3 * n * case["rot"]}
    if case["op"] == "append":
        held, new = _held(case)
        n = sum(new) * case["Hk"] * d * 2
        return {"bytes": 3 * n, "flops": 2 * n}
    lens, live = _lengths(case)
    total_bytes, flops = 0, 0
    for n, q in zip(lens, live):
        keys = n
        if case["mask"] == "window":
            keys = min(n, case["window"] + case["prefix"] + q - 1)
        elif case["mask"] == "documents":
            keys = min(n, (n - 1) % max(case["window"], 1) + q)
        total_bytes += 2 * keys * case["Hk"] * d + 4 * q * case["H"] * d + 4 * q * case["H"]
        flops += 4 * q * case["H"] * d * max(1, keys - (0 if case["mask"] == "all" else q // 2))
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


def _table(B, pages_each, gen, dev):
    """A page table whose pages lie in random order, and the number of pages. Entries
    behind a sequence's last page are -1, as a server that maps pages late has them."""
    most, total = max(pages_each), sum(pages_each)
    order = torch.randperm(total, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    need = torch.tensor(pages_each, device=dev)
    at = torch.cumsum(need, 0) - need
    col = torch.arange(most, device=dev)
    live = col[None, :] < need[:, None]
    idx = torch.where(live, at[:, None] + col[None, :], 0)
    return torch.where(live, order[idx], -1).to(torch.int32).contiguous(), total


def _cache(pages, Hk, d, gen, dev):
    """A filled cache: normal values at scales that differ from page to page."""
    s = {}
    for name, shape in (("k", (pages, Hk, PAGE, d)), ("v", (pages, Hk, d, PAGE))):
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        step = max(1, (1 << 27) // (Hk * PAGE * d))
        for p in range(0, pages, step):
            x = torch.randn((min(step, pages - p),) + shape[1:], generator=gen, device=dev)
            codes[p:p + step] = (x * 96.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        k = torch.randint(-8, -5, (pages, Hk), generator=gen, device=dev)
        s[name + "8"] = codes
        s[name + "scale"] = torch.exp2(k.float())
    return s


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, N, d = case["B"], case["N"], case["d"]
    state = {"case": case, "op": case["op"]}
    randn = lambda shape, dt=torch.bfloat16: torch.randn(shape, generator=gen, device=dev).to(dt)
    if case["op"] == "rope":
        Hq, Hk, dt = case["Hq"], case["Hk"], DTYPES[case["dtype"]]
        if case["strided"]:  # slices of a fused projection, token-major
            x = randn((B, N, (Hq + 2 * Hk) * d), dt)
            q = x[..., :Hq * d].unflatten(2, (Hq, d)).transpose(1, 2)
            k = x[..., Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d)).transpose(1, 2)
        else:
            q, k = randn((B, Hq, N, d), dt), randn((B, Hk, N, d), dt)
        f, c = _frequencies(case["rot"], case["scaling"])
        t = torch.arange(N, device=dev)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=dev)
        span = -(-N // case["docs"])
        state.update(q=q, k=k, freqs=torch.tensor(f, dtype=torch.float64).to(dev), c=c,
                     positions=(first + t % span).to(torch.int32).contiguous())
        return state
    if case["op"] == "append":
        Hk = case["Hk"]
        held, new = _held(case)
        pages_each = [-(-(h + n) // PAGE) for h, n in zip(held, new)]
        table, pages = _table(B, pages_each, gen, dev)
        state.update(_cache(pages, Hk, d, gen, dev), table=table,
                     k=randn((B, Hk, N, d)) * 2, v=randn((B, Hk, N, d)),
                     start=torch.tensor(held, dtype=torch.int32, device=dev),
                     count=torch.tensor(new, dtype=torch.int32, device=dev))
    else:
        H, Hk = case["H"], case["Hk"]
        lens, live = _lengths(case)
        table, pages = _table(B, [-(-n // PAGE) for n in lens], gen, dev)
        state.update(_cache(pages, Hk, d, gen, dev), table=table, q=randn((B, H, N, d)),
                     lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                     live=torch.tensor(live, dtype=torch.int32, device=dev),
                     o=torch.zeros((B, H, N, d), dtype=torch.bfloat16, device=dev),
                     lse=torch.zeros((B, H, N), device=dev), lts=None, lte=None,
                     causal=case["mask"] != "all")
        if case["mask"] in ("window", "documents"):
            L, Hm, w = table.shape[1] * PAGE, case["Hm"], case["window"]
            j = torch.arange(L, device=dev, dtype=torch.int32)
            h = torch.arange(Hm, device=dev, dtype=torch.int32)[:, None]
            if case["mask"] == "window":
                lts = torch.where(j[None] < case["prefix"], L, (j[None] + w - h % w).clamp(max=L))
            else:
                lts = ((j[None] // w + 1) * w).clamp(max=L).expand(Hm, L)
            state["lts"] = lts[None].expand(B, Hm, L).to(torch.int32).contiguous()
            state["lte"] = torch.full_like(state["lts"], L)
    if own:
        from mask_aware_exact_gb300 import flashmask as fm
        state["cache"] = fm.KVCache(state["k8"], state["v8"], state["kscale"], state["vscale"])
        if case["op"] == "append":
            state["ws"] = fm.alloc_cache_workspace(B, case["Hk"], case["Hk"], N, d,
                                                   state["table"].shape[1])
        else:
            state["mask"] = fm.DeviceMask(state["lts"], state["lte"], None, None, state["causal"])
            state["ws"] = fm.alloc_cache_workspace(B, case["H"], case["Hk"], N, d,
                                                   state["table"].shape[1])
    return state


# ---------------------------------------------------------------- plain forms
def _rope_plain(s):
    case = s["case"]
    n, rot = case["rot"] // 2, case["rot"]
    a = s["positions"].double()[:, None, :, None] * s["freqs"]
    if case["backward"]:
        a = -a
    cos, sin = (torch.cos(a) * s["c"]).float(), (torch.sin(a) * s["c"]).float()
    out = {}
    for name in ("q", "k"):
        x = s[name]
        xf = x[..., :rot].float()
        x0, x1 = (xf[..., 0::2], xf[..., 1::2]) if case["interleaved"] else (xf[..., :n], xf[..., n:])
        y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
        y = torch.stack((y0, y1), -1).flatten(-2) if case["interleaved"] else torch.cat((y0, y1), -1)
        out[name] = torch.cat((y.to(x.dtype), x[..., rot:]), -1)
    return out


def _gather(codes, scale, table):
    """[B, M, Hk, ...] values of the pages in `table` (entries below 0 read page 0)."""
    t = table.clamp(min=0).long()
    return codes.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]


def _scale_of(absmax):
    m, e = torch.frexp(absmax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-100)
    k = torch.where(absmax > 0, k, -100)
    return torch.ldexp(torch.ones_like(absmax), k)


def _append_plain(s):
    case = s["case"]
    B, Hk, N, d = case["B"], case["Hk"], case["N"], case["d"]
    dev, table = s["k"].device, s["table"]
    start, count = s["start"].long(), s["count"].long()
    W = (N + PAGE - 2) // PAGE + 1
    slot = torch.arange(W * PAGE, device=dev)[None] - start[:, None] % PAGE  # new token of a slot
    new = ((slot >= 0) & (slot < count[:, None])).view(B, W, 1, PAGE)
    token = slot.clamp(0, N - 1)
    before = (slot < 0).view(B, W, 1, PAGE)
    fresh = torch.ones((B, W), dtype=torch.bool, device=dev)
    fresh[:, 0] = start % PAGE == 0
    touched = new.any(-1)[:, :, 0]
    col = (start[:, None] // PAGE + torch.arange(W, device=dev)).clamp(max=table.shape[1] - 1)
    page = torch.where(touched, torch.gather(table.long(), 1, col), 0)
    for x, name in ((s["k"], "k"), (s["v"], "v")):
        x = torch.gather(x.float(), 2, token[:, None, :, None].expand(B, Hk, W * PAGE, d))
        x = x.view(B, Hk, W, PAGE, d).transpose(1, 2) * new[..., None]  # [B, W, Hk, 64, d]
        held = s[name + "8"].view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
        if name == "v":
            held = held.transpose(-1, -2)
        was = s[name + "scale"][page]  # [B, W, Hk]
        need = _scale_of(x.abs().amax((-1, -2)))
        scale = torch.where(fresh[..., None], need, torch.maximum(need, was))
        kept = torch.where(before[..., None], held * (was / scale)[..., None, None],
                           torch.where(fresh[..., None, None, None], 0.0, held))
        codes = torch.where(new[..., None], x / scale[..., None, None], kept).to(torch.float8_e4m3fn)
        if name == "v":
            codes = codes.transpose(-1, -2)
        s[name + "8"].view(torch.uint8)[page[touched]] = codes.view(torch.uint8)[touched]
        s[name + "scale"][page[touched]] = scale[touched]
    return {n: s[n] for n in ("k8", "kscale", "v8", "vscale")}


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


def _attend_plain(s):
    case = s["case"]
    B, H, Hk, N, d = (case[n] for n in ("B", "H", "Hk", "N", "d"))
    G, L = H // Hk, s["table"].shape[1] * PAGE
    k = _gather(s["k8"], s["kscale"], s["table"]).transpose(1, 2).reshape(B, Hk, L, d)
    score = s["q"].float().view(B, Hk, G * N, d) @ k.transpose(-1, -2)
    del k
    score = score.view(B, H, N, L).mul_(1.0 / math.sqrt(d))
    see = _visible(s, torch.arange(L, device=score.device), torch.arange(N, device=score.device))
    if see.shape[1] > 1:
        see = see.repeat_interleave(H // see.shape[1], 1)
    score.masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _gather(s["v8"], s["vscale"], s["table"]).permute(0, 2, 1, 4, 3).reshape(B, Hk, L, d)
    o = (p.view(B, Hk, G * N, L) @ v).view(B, H, N, d) / total.clamp(min=1e-37)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    live = (torch.arange(N, device=o.device) < s["live"][:, None])[:, None]
    return {"o": torch.where(live[..., None], o.to(torch.bfloat16), s["o"]),
            "lse": torch.where(live, lse, s["lse"])}


def run(state):
    op = state["op"]
    if own:
        from mask_aware_exact_gb300 import flashmask as fm
        if op == "rope":
            rope = fm.flashmask_rope_bwd if state["case"]["backward"] else fm.flashmask_rope
            q, k = rope(state["q"], state["k"], state["freqs"], positions=state["positions"],
                        interleaved=state["case"]["interleaved"], mscale=state["c"])
            return {"q": q, "k": k}
        if op == "append":
            fm.flashmask_cache_append(state["cache"], state["table"], state["k"], state["v"],
                                      state["start"], state["ws"], count=state["count"])
            return {n: state[n] for n in ("k8", "kscale", "v8", "vscale")}
        o, lse = fm.flashmask_fwd_cache(state["q"], state["cache"], state["table"], state["lens"],
                                        state["ws"], mask=state["mask"], q_lens=state["live"],
                                        o=state["o"], lse=state["lse"])
        return {"o": o, "lse": lse}
    return {"rope": _rope_plain, "append": _append_plain, "attend": _attend_plain}[op](state)


# ---------------------------------------------------------------- 64-bit results
def _exact_rope(s):
    case, out = s["case"], {}
    rot = case["rot"]
    i = torch.arange(rot // 2, device=s["q"].device)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    angle = torch.einsum("bn,i->bni", s["positions"].double(), s["freqs"])
    turn = torch.polar(torch.full_like(angle, s["c"]), -angle if case["backward"] else angle)
    for name in ("q", "k"):
        y = s[name].double().clone(memory_format=torch.contiguous_format)
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _round_e4m3(x):
    """Nearest e4m3 value (ties to even) of 64-bit values of magnitude <= 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _exact_append(s):
    out = {}
    table, held, new = (s[n].tolist() for n in ("table", "start", "count"))
    for name in ("k", "v"):
        codes, scales = s[name + "8"].double(), s[name + "scale"].double()
        for b in range(len(held)):
            t, end = held[b], held[b] + new[b]
            while t < end:
                page, lo = table[b][t // PAGE], t % PAGE
                n = min(PAGE - lo, end - t)
                x = s[name][b, :, t - held[b]:t - held[b] + n].double()  # [Hk, n, d]
                body = codes[page] if name == "k" else codes[page].transpose(-1, -2)
                top = x.abs().amax((1, 2))
                k = torch.ceil(torch.log2(top / 448.0))
                k = k + (top > 448.0 * torch.exp2(k)).double() - (top <= 224.0 * torch.exp2(k)).double()
                scale = torch.exp2(k.clamp(min=-100.0))
                if lo:
                    scale = torch.maximum(scale, scales[page])
                    body[:, :lo] = _round_e4m3(body[:, :lo] * (scales[page] / scale)[:, None, None])
                else:
                    body[:, n:] = 0.0
                body[:, lo:lo + n] = _round_e4m3(x / scale[:, None, None])
                scales[page] = scale
                t += n
        out[name + "8"], out[name + "scale"] = codes, scales
    return {n: out[n] for n in ("k8", "kscale", "v8", "vscale")}


def _exact_attend(s):
    case = s["case"]
    H, Hk, N, d = (case[n] for n in ("H", "Hk", "N", "d"))
    o, lse = s["o"].double(), s["lse"].double()
    for b, (n, live) in enumerate(zip(s["lens"].tolist(), s["live"].tolist())):
        pages = s["table"][b, :-(-n // PAGE)].long()
        j = torch.arange(n, device=o.device)
        pos = torch.arange(n - live, n, device=o.device)[:, None]
        for h in range(H):
            hk = h // (H // Hk)
            k = s["k8"][pages, hk].double() * s["kscale"][pages, hk].double()[:, None, None]
            v = s["v8"][pages, hk].double() * s["vscale"][pages, hk].double()[:, None, None]
            k, v = k.reshape(-1, d)[:n], v.transpose(1, 2).reshape(-1, d)[:n]
            x = s["q"][b, h, :live].double() @ k.T / math.sqrt(d)
            hidden = (j > pos) if s["causal"] else torch.zeros_like(x, dtype=torch.bool)
            if s["lts"] is not None:
                m = h // (H // s["lts"].shape[1])
                hidden = hidden | ((s["lts"][b, m, :n] <= pos) & (pos < s["lte"][b, m, :n]))
            x = x.masked_fill(hidden, -math.inf)
            total = torch.logsumexp(x, -1)
            lse[b, h, :live] = total
            o[b, h, :live] = torch.where(torch.isinf(total)[:, None], 0.0,
                                         torch.exp(x - total[:, None])) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[s["op"]](s)
