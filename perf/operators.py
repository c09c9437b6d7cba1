"""Operators around a paged key/value cache: what is measured, and their plain forms.

The serving path of the attention library: rotary positions on the new queries
and keys (``rope``), the new keys and values written into the pages of a cache,
held as BF16 or quantised to E4M3 (``cache_write``), pages read back as packed
BF16 rows (``cache_read``), and attention of the new tokens over the pages
(``fwd_paged``).

A quantised row (one token, one head, D values) is held as D E4M3 codes and one
power-of-two scale 2^e, e the smallest exponent in [-110, 119] with
amax <= 448 * 2^e, stored as the byte e + 127.  A row that holds a NaN or an
infinity has the byte 255 and stands for NaN.

Shapes: q [B, n, Hq, D] or packed [total, Hq, D]; pages
[num_pages, Hkv, page_size, D]; scales [num_pages, Hkv, page_size]; block_table
[B, pages per sequence], entries behind a sequence's last page unused; seq_lens
[B] count the keys of each sequence, its new tokens among them.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
E_MIN, E_MAX = -110, 119
ROPE_BASE = 10000.0


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one new token of each of 64 sequences, three axes (time, height, width) as in a decoding step
        dict(name="rope_step", op="rope", B=64, n=1, Hq=32, Hkv=8, D=128, axes=3, rot=64, restart=False,
             interleaved=False, inverse=False, far=200000),
        # gradients of a training step's queries and keys: the rotation backwards, frequencies restarting on each axis
        dict(name="rope_train_back", op="rope", B=2, n=8192, Hq=16, Hkv=16, D=128, axes=3, rot=64, restart=True,
             interleaved=False, inverse=True, far=4096),
        # an odd packed prompt, D = 64, adjacent pairs, part of the head rotated, one axis
        dict(name="rope_prompt_d64", op="rope", B=1, n=4099, Hq=16, Hkv=2, D=64, axes=1, rot=24, restart=False,
             interleaved=True, inverse=False, far=262143),
        # a decoding step's new keys and values quantised into the cache: the smallest call
        dict(name="write_step_e4m3", op="write", B=64, n=1, ragged=False, Hkv=8, D=128, page=16, past=2048,
             e4m3=True, lens=1),
        # ragged prompts of a prefill quantised as they are written
        dict(name="write_prompts_e4m3", op="write", B=13, n=2500, ragged=True, Hkv=8, D=128, page=64, past=700,
             e4m3=True, lens=2),
        # a long prompt written as BF16, D = 64
        dict(name="write_prompt_bf16_d64", op="write", B=1, n=32768, ragged=False, Hkv=16, D=64, page=128, past=1,
             e4m3=False, lens=3),
        # a quantised cache of ragged sequences read back, for dense attention or a move to another cache
        dict(name="read_e4m3", op="read", B=24, L=8192, Hkv=8, D=128, page=32, e4m3=True, lens=4),
        # a short odd BF16 cache read back
        dict(name="read_bf16_d64", op="read", B=3, L=333, Hkv=4, D=64, page=16, e4m3=False, lens=5),
        # one user, one new token, a short cache: latency counts
        dict(name="decode_single_bf16", op="attn", B=1, n=1, ragged=False, Hq=32, Hkv=8, D=128, page=16, L=1023,
             e4m3=False, causal=True, lens=6),
        # a decoding step of 64 ragged sequences over a quantised cache
        dict(name="decode_batch_e4m3", op="attn", B=64, n=1, ragged=False, Hq=32, Hkv=8, D=128, page=64, L=8192,
             e4m3=True, causal=True, lens=2),
        # a long prompt's chunk over 30 K cached keys
        dict(name="chunk_long_bf16", op="attn", B=1, n=2048, ragged=False, Hq=32, Hkv=8, D=128, page=128, L=32768,
             e4m3=False, causal=True, lens=7),
        # ragged chunks and single tokens in one call over a quantised cache
        dict(name="chunk_mixed_e4m3", op="attn", B=12, n=500, ragged=True, Hq=16, Hkv=4, D=128, page=32, L=9000,
             e4m3=True, causal=True, lens=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8), (16, 16), (16, 4), (16, 2), (8, 1), (24, 8), (40, 8), (28, 4), (4, 4)]
PAGES = [16, 32, 64, 128, 256]


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn"])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128])
    c = dict(op=op, Hkv=Hkv, D=D)
    if op == "rope":
        B = _log(rng, 1, 64)
        n = max(1, min(_log(rng, 1, 16384), 33554432 // (B * (Hq + Hkv) * D)))
        axes = rng.choice([1, 2, 3])
        c.update(B=B, n=n, Hq=Hq, axes=axes, rot=rng.randint(max(axes, D // 8), D // 2), restart=rng.random() < 0.5,
                 interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, far=_log(rng, 64, 262143))
        return c
    c.update(page=rng.choice(PAGES), e4m3=rng.random() < 0.6, lens=rng.randint(0, 10 ** 6))
    if op == "write":
        B = _log(rng, 1, 128)
        n = max(1, min(_log(rng, 1, 32768), 33554432 // (B * Hkv * D)))
        past = max(0, min(_log(rng, 1, 8192) - 1, 67108864 // (B * Hkv * D) - n))
        c.update(B=B, n=n, ragged=rng.random() < 0.5, past=past)
    elif op == "read":
        B = _log(rng, 1, 64)
        c.update(B=B, L=max(1, min(_log(rng, 16, 65536), 201326592 // (B * Hkv * D))))
    else:
        long = rng.random() < 0.5
        B = _log(rng, 1, 16 if long else 128)
        n = _log(rng, 17, 2048) if long else rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        L = max(n, min(_log(rng, 16, 65536), 536870912 // (B * Hkv * D)))
        n = max(1, min(n, 1073741824 // (B * Hq * L)))
        c.update(B=B, n=n, ragged=rng.random() < 0.5, Hq=Hq, L=L, causal=rng.random() < 0.8)
    return c


def _lengths(c):
    """(new tokens, keys) of every sequence.  The longest sequence is the first."""
    r = random.Random(c["lens"])
    B = c["B"]
    if c["op"] == "read":
        keys = [c["L"]] + [r.randint(1, c["L"]) for _ in range(B - 1)]
        return [0] * B, keys
    n = c["n"]
    # ragged: half of the other sequences take one new token, the rest up to n
    new = [n] + [(1 if r.random() < 0.5 else r.randint(1, n)) if c["ragged"] else n for _ in range(B - 1)]
    if c["op"] == "write":
        keys = [m + r.randint(0, c["past"]) for m in new]
    else:
        lo = min(128, c["L"])
        keys = [c["L"]] + [max(m, r.randint(lo, c["L"])) for m in new[1:]]
    return new, keys


def _sections(c):
    """Rotary pairs of each axis: as equal as they go."""
    a, rot = c["axes"], c["rot"]
    return [rot // a + (1 if i < rot % a else 0) for i in range(a)]


# ------------------------------------------------------------------ inputs --

def _quantise(x):
    """E4M3 codes (as float8 values) and scale bytes of rows x [..., D]."""
    x = x.float()
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    m, k = torch.frexp(torch.where(bad, torch.zeros_like(amax), amax))     # amax = m * 2^k, 0.5 <= m < 1
    e = torch.where(m <= 0.875, k - 9, k - 8)                              # 448 = 0.875 * 2^9
    e = torch.where(amax == 0, torch.full_like(e, E_MIN), e).clamp(E_MIN, E_MAX)
    y = torch.ldexp(x, -e.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    codes = torch.where(bad.unsqueeze(-1), torch.zeros_like(y), y).to(torch.float8_e4m3fn)
    return codes, torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _value(codes, scale):
    """FP32 values that codes and scale bytes stand for."""
    f = torch.ldexp(torch.ones((), device=codes.device), scale.int() - 127)
    f = torch.where(scale == 255, torch.full_like(f, math.nan), f)
    return codes.float() * f.unsqueeze(-1)


def _randn(shape, g, spread=False):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if spread:   # channels of unlike size, as keys have them
        x = x * torch.exp(0.7 * torch.randn(shape[-1], generator=g, device="cuda")).to(torch.bfloat16)
    return x


def _cache(c, keys, g):
    """Pages, scales (or None), block table: every sequence's keys in shuffled pages, spare pages between them."""
    P, Hkv, D = c["page"], c["Hkv"], c["D"]
    counts = [-(-k // P) for k in keys]
    total, spare = sum(counts), 3
    order = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor([sum(counts[:i]) for i in range(len(counts))], device="cuda")
    cols = torch.arange(max(counts), device="cuda")
    at = (start.unsqueeze(1) + cols).clamp(max=total + spare - 1)
    used = cols < torch.tensor(counts, device="cuda").unsqueeze(1)
    table = torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous()
    s = {"block_table": table}
    for name in ("k", "v"):
        pages = _randn((total + spare, Hkv, P, D), g, spread=name == "k")
        if c["e4m3"]:
            flat = pages.view(-1, D)
            codes = torch.empty(flat.shape, dtype=torch.float8_e4m3fn, device="cuda")
            scale = torch.empty(flat.shape[0], dtype=torch.uint8, device="cuda")
            for i in range(0, flat.shape[0], 1 << 20):
                codes[i:i + (1 << 20)], scale[i:i + (1 << 20)] = _quantise(flat[i:i + (1 << 20)])
            s[name + "_pages"], s[name + "_scale"] = codes.view(pages.shape), scale.view(pages.shape[:-1])
        else:
            s[name + "_pages"], s[name + "_scale"] = pages, None
    return s


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "rope":
        shape = (c["B"], c["n"])
        pos = torch.randint(0, c["far"] + 1, (c["axes"],) + shape, generator=g, device="cuda", dtype=torch.int32)
        return {"case": c, "q": _randn(shape + (c["Hq"], D), g), "k": _randn(shape + (Hkv, D), g), "pos": pos}
    new, keys = _lengths(c)
    s = _cache(c, keys, g)
    s.update(case=c, keys=torch.tensor(keys, dtype=torch.int32, device="cuda"), max_k=max(keys))
    if c["op"] == "read":
        s.update(cu=_cu(keys), total=sum(keys))
        return s
    ragged = c["ragged"]
    lead = (sum(new),) if ragged else (c["B"], c["n"])
    s.update(cu=_cu(new) if ragged else None, max_q=max(new))
    if c["op"] == "write":
        s.update(k=_randn(lead + (Hkv, D), g, spread=True), v=_randn(lead + (Hkv, D), g))
    else:
        s.update(q=_randn(lead + (c["Hq"], D), g))
    return s


# ------------------------------------------------------------- plain forms --

def _inv_freq(c):
    """(axis of each rotary pair, its frequency), on the host."""
    sec, out = _sections(c), []
    for a, m in enumerate(sec):
        first = len(out)
        out += [(a, ROPE_BASE ** (-(i / m if c["restart"] else (first + i) / c["rot"]))) for i in range(m)]
    return [a for a, _ in out], [f for _, f in out]


def _rope_plain(s):
    c = s["case"]
    axis, freq = _inv_freq(c)
    axis = torch.tensor(axis, device="cuda")
    freq = torch.tensor(freq, device="cuda", dtype=torch.float64)
    ang = s["pos"].double()[axis].movedim(0, -1) * freq            # [B, n, pairs]; far positions need 64 bits
    cos, sin = ang.cos().float().unsqueeze(-2), ang.sin().float().unsqueeze(-2)
    if c["inverse"]:
        sin = -sin
    rot = c["rot"]

    def turn(x):
        x = x.float()
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:2 * rot:2], x[..., 1:2 * rot:2]
            y[..., 0:2 * rot:2], y[..., 1:2 * rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot], x[..., rot:2 * rot]
            y[..., :rot], y[..., rot:2 * rot] = a * cos - b * sin, b * cos + a * sin
        return y.to(torch.bfloat16)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _token_slots(cu, lens, total, table, page):
    """(page, slot in it) of packed tokens cu[b] .. cu[b+1], the last cu[b+1] - cu[b] of lens[b]."""
    i = torch.arange(total, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu[1:], i, right=True)
    pos = lens[b] - (cu[b + 1] - i)
    return table[b, (pos // page).long()].long(), (pos % page).long()


def _write_plain(s):
    c = s["case"]
    D, Hkv = c["D"], c["Hkv"]
    cu = s["cu"]
    if cu is None:
        cu = torch.arange(c["B"] + 1, device="cuda", dtype=torch.int32) * c["n"]
    out = {}
    for name in ("k", "v"):
        x = s[name].view(-1, Hkv, D)
        page, slot = _token_slots(cu, s["keys"], x.shape[0], s["block_table"], c["page"])
        pages, scale = s[name + "_pages"], s[name + "_scale"]
        if c["e4m3"]:
            codes, e = _quantise(x)
            pages.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            scale[page, :, slot] = e
            out[name + "_scale"] = scale
        else:
            pages[page, :, slot] = x
        out[name + "_pages"] = pages
    return out


def _read_plain(s):
    c = s["case"]
    out = {}
    page, slot = _token_slots(s["cu"], s["keys"], s["total"], s["block_table"], c["page"])
    for name in ("k", "v"):
        if c["e4m3"]:
            codes = s[name + "_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
            out[name] = _value(codes, s[name + "_scale"][page, :, slot]).to(torch.bfloat16)
        else:
            out[name] = s[name + "_pages"][page, :, slot]
    return out


def _attn_plain(s):
    c = s["case"]
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    n, L, grp = s["max_q"], s["max_k"], Hq // Hkv
    table = s["block_table"].clamp(min=0).long()

    def gather(name):     # [B, Hkv, keys, D], padded to the longest sequence
        pages = s[name + "_pages"]
        if c["e4m3"]:
            x = _value(pages.view(torch.uint8)[table].view(torch.float8_e4m3fn), s[name + "_scale"][table])
        else:
            x = pages[table].float()
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :L]

    row = torch.arange(n, device="cuda")
    if s["cu"] is None:
        q = s["q"]
        new = torch.full((B,), n, device="cuda")
    else:                 # padded to the most new tokens of any sequence
        new = (s["cu"][1:] - s["cu"][:-1]).long()
        at = (s["cu"][:-1].long().unsqueeze(1) + row).clamp(max=s["q"].shape[0] - 1)
        q = s["q"][at]
    q = q.float().reshape(B, n, Hkv, grp, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, grp * n, D)
    x = (q @ gather("k").transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, grp, n, L)
    key = torch.arange(L, device="cuda")
    last = s["keys"].long().view(B, 1, 1) - 1                         # the last key a row sees
    last = last - (new.view(B, 1, 1) - 1 - row.view(1, n, 1)) if c["causal"] else last.expand(B, n, 1)
    x.masked_fill_((key > last).view(B, 1, 1, n, L), -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, grp * n, L) @ gather("v")).view(B, Hkv, grp, n, D)
    o = (o / l.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(torch.bfloat16)
    lse = (m + l.log()).view(B, Hq, n)
    if s["cu"] is None:
        return {"o": o, "lse": lse}
    b = torch.searchsorted(s["cu"][1:].long(), torch.arange(s["q"].shape[0], device="cuda"), right=True)
    r = torch.arange(s["q"].shape[0], device="cuda") - s["cu"][b]
    return {"o": o[b, r], "lse": lse[b, :, r].t().contiguous()}


# --------------------------------------------------------------------- run --

def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"rope": _rope_plain, "write": _write_plain, "read": _read_plain, "attn": _attn_plain}[c["op"]](s)
    import exact_attention_78_gb300 as fa

    if c["op"] == "rope":
        q, k = fa.rope(s["q"], s["k"], s["pos"], sections=_sections(c), base=ROPE_BASE, restart=c["restart"],
                       interleaved=c["interleaved"], inverse=c["inverse"])
        return {"q": q, "k": k}
    quant = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["op"] == "write":
        fa.cache_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["keys"], cu_seqlens=s["cu"],
                       **quant)
        return {x: s[x] for x in ("k_pages", "v_pages") + (("k_scale", "v_scale") if c["e4m3"] else ())}
    if c["op"] == "read":
        k, v = fa.cache_read(s["k_pages"], s["v_pages"], s["block_table"], s["cu"], s["total"], **quant)
        return {"k": k, "v": v}
    o, lse = fa.fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["keys"], causal=c["causal"],
                          cu_seqlens=s["cu"], max_q=s["max_q"], **quant)
    return {"o": o, "lse": lse}


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "rope":
        t = c["B"] * c["n"]
        h = c["Hq"] + Hkv
        return {"bytes": 2 * t * h * D * 2 + 4 * t * c["axes"], "flops": 6 * t * h * c["rot"]}
    new, keys = _lengths(c)
    held = (D + 1 if c["e4m3"] else 2 * D) * Hkv * 2       # bytes of one token's key and value in the cache
    plain = 2 * D * Hkv * 2
    pages = 4 * sum(-(-k // c["page"]) for k in keys)
    if c["op"] == "write":
        return {"bytes": sum(new) * (held + plain) + 4 * sum(-(-n // c["page"]) for n in new),
                "flops": 2 * sum(new) * Hkv * D * 2}
    if c["op"] == "read":
        return {"bytes": sum(keys) * (held + plain) + pages, "flops": sum(keys) * Hkv * D * 2}
    seen = sum(n * k - (n * (n - 1) // 2 if c["causal"] else 0) for n, k in zip(new, keys))
    return {"bytes": sum(keys) * held + pages + sum(new) * c["Hq"] * (4 * D + 4), "flops": 4 * seen * c["Hq"] * D}


# ------------------------------------------------------------------- exact --

def _exact_write(s, new, keys):
    """The pages after the write: the codes' values (their scale taken out) or the BF16 values."""
    c = s["case"]
    P, D = c["page"], c["D"]
    out = {}
    for name in ("k", "v"):
        pages = s[name + "_pages"].double()
        x = s[name].reshape(-1, c["Hkv"], D).double()
        if c["e4m3"]:
            amax = x.abs().amax(-1, keepdim=True)
            e = torch.floor(torch.log2(amax.clamp(min=1e-300))) - 8      # 2^(e+8) <= amax: too small by one if
            e = e + (amax > E4M3_MAX * torch.exp2(e)).double()           # amax is above 448 * 2^e
            y = x / torch.exp2(e.clamp(E_MIN, E_MAX))
            y = y.clamp(-E4M3_MAX, E4M3_MAX)
            # four significant bits, steps of 2^-9 below 2^-6; ties to even
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(y / step) * step
        first = 0
        for n, L, table in zip(new, keys, s["block_table"].tolist()):
            for t in range(L - n, L, P):       # a page's worth of new tokens at a time, over at most two pages
                at = torch.arange(t, min(t + P, L), device="cuda")
                page = torch.tensor([table[t // P], table[min(t + P - 1, L - 1) // P]], device="cuda")
                pages[page[at // P - t // P], :, at % P] = x[first + t - (L - n) + torch.arange(len(at), device="cuda")]
            first += n
        out[name + "_pages"] = pages
        if c["e4m3"]:
            out[name + "_scale"] = None
    return out


def exact(case, seed):
    """The definitions in 64 bits, one sequence (and key/value head) at a time."""
    c = case
    s = prepare(c, seed)
    D, Hkv, P = c["D"], c["Hkv"], c.get("page")
    if c["op"] == "rope":
        sec = _sections(c)
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            i = 0
            for a, m in enumerate(sec):
                for j in range(m):
                    t = s["pos"][a].double() / ROPE_BASE ** (j / m if c["restart"] else i / c["rot"])
                    z = torch.polar(torch.ones_like(t), -t if c["inverse"] else t).unsqueeze(-1)
                    one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"])
                    w = torch.complex(x[..., one], x[..., two]) * z
                    y[..., one], y[..., two] = w.real, w.imag
                    i += 1
            out[name] = y
        return out
    new, keys = _lengths(c)
    if c["op"] == "write":
        return _exact_write(s, new, keys)

    def rows(name, b):    # keys or values of sequence b, [L, Hkv, D] in 64 bits
        at = torch.arange(keys[b], device="cuda")
        page, slot = s["block_table"][b][at // P].long(), at % P
        if not c["e4m3"]:
            return s[name + "_pages"][page, :, slot].double()
        codes = s[name + "_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).double()
        return codes * torch.exp2(s[name + "_scale"][page, :, slot].double() - 127.0).unsqueeze(-1)

    if c["op"] == "read":
        return {x: torch.cat([rows(x, b) for b in range(c["B"])]) for x in ("k", "v")}
    if work(c)["flops"] > 2.5e12:
        return None
    grp = c["Hq"] // Hkv
    o_all, l_all, first = [], [], 0
    for b in range(c["B"]):
        n, L = new[b], keys[b]
        q = (s["q"][b] if s["cu"] is None else s["q"][first:first + n]).double()
        first += n
        k, v = rows("k", b), rows("v", b)
        o = torch.empty(n, c["Hq"], D, dtype=torch.float64, device="cuda")
        lse = torch.empty(c["Hq"], n, dtype=torch.float64, device="cuda")
        hidden = None
        if c["causal"] and n > 1:
            hidden = torch.ones(n, L, dtype=torch.bool, device="cuda").triu(L - n + 1)
        for h in range(c["Hq"]):
            x = q[:, h] @ k[:, h // grp].T / math.sqrt(D)
            if hidden is not None:
                x = x.masked_fill(hidden, -math.inf)
            lse[h] = torch.logsumexp(x, -1)
            o[:, h] = torch.exp(x - lse[h].unsqueeze(-1)) @ v[:, h // grp]
        o_all.append(o)
        l_all.append(lse)
    if s["cu"] is None:
        return {"o": torch.stack(o_all), "lse": torch.stack(l_all)}
    return {"o": torch.cat(o_all), "lse": torch.cat(l_all, 1)}
