"""Operators of speculative decoding and of eviction over a paged cache: what is measured, and their plain forms.

Speculative decoding: ``tree_mask`` makes, from the parents of a tree of drafted
tokens, which drafted tokens each of them sees and how deep it lies;
``fwd_paged`` with ``tree`` attends from all drafted tokens to the cache and to
their ancestors; ``cache_keep`` moves the accepted ones' rows to the front.

Eviction: ``cache_weights`` adds up, key by key, the attention weight that the
new tokens give to it; ``cache_select`` chooses which tokens of a sequence each
key/value head keeps by those sums; ``cache_keep`` moves the kept rows together.

A quantised row (one token, one head, D values) is held as D E4M3 codes and one
power-of-two scale 2^e, stored as the byte e + 127.

Shapes: q [B, n, Hq, D] or packed [total, Hq, D]; pages
[num_pages, Hkv, page_size, D]; scales and sums [num_pages, Hkv, page_size];
block_table [B, pages per sequence], entries behind a sequence's last page
unused; seq_lens [B] count the keys of each sequence, its new tokens among them.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
E_MIN, E_MAX = -110, 119


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one user's tree of drafts: the smallest call
        dict(name="mask_single", op="mask", B=1, n=25, ragged=False, lens=1),
        # a batch's ragged trees, packed, some of them wide
        dict(name="mask_batch_packed", op="mask", B=256, n=200, ragged=True, lens=2),
        # one user, a tree of 25 drafted tokens over a short cache: latency counts
        dict(name="tree_single_bf16", op="attn", B=1, n=25, ragged=False, Hq=32, Hkv=8, D=128, page=16, L=2047,
             e4m3=False, lens=3),
        # a batch's ragged trees over a quantised cache
        dict(name="tree_batch_e4m3", op="attn", B=48, n=61, ragged=True, Hq=32, Hkv=8, D=128, page=64, L=8192,
             e4m3=True, lens=4),
        # small trees of a batch, a key/value head for each query head, D = 64
        dict(name="tree_few_bf16_d64", op="attn", B=64, n=7, ragged=False, Hq=16, Hkv=16, D=64, page=32, L=4096,
             e4m3=False, lens=5),
        # a decoding step of 64 ragged sequences over a quantised cache, whose keys' weights are added up
        dict(name="weigh_step_e4m3", op="weigh", B=64, n=1, ragged=False, Hq=32, Hkv=8, D=128, page=64, L=8192,
             e4m3=True, causal=True, decay=1.0, lens=6),
        # ragged chunks and single tokens over a short BF16 cache, D = 64, older sums fading
        dict(name="weigh_mixed_bf16_d64", op="weigh", B=10, n=150, ragged=True, Hq=16, Hkv=4, D=64, page=16, L=3001,
             e4m3=False, causal=True, decay=0.97, lens=7),
        # a long prompt's last chunk, by whose weights the prompt's keys are to be evicted
        dict(name="weigh_prompt_bf16", op="weigh", B=1, n=2048, ragged=False, Hq=32, Hkv=8, D=128, page=128, L=32768,
             e4m3=False, causal=True, decay=1.0, lens=8),
        # a batch of ragged sequences brought down to a budget of 2048 tokens for each head
        dict(name="select_batch", op="select", B=24, Hkv=8, page=64, L=12000, keep=2048, first=4, recent=256, lens=9),
        # one long sequence
        dict(name="select_long", op="select", B=1, Hkv=4, page=16, L=200001, keep=16000, first=16, recent=1000,
             lens=10),
        # that batch's kept rows moved together, each head its own, in a quantised cache with its sums
        dict(name="keep_evicted_e4m3", op="keep", B=24, Hkv=8, D=128, page=64, L=12000, keep=2048, first=4,
             recent=256, path=False, e4m3=True, lens=9),
        # accepted drafts of a decoding step, all heads alike
        dict(name="keep_accepted_bf16", op="keep", B=48, Hkv=8, D=128, page=32, L=4096, keep=6, first=0, recent=0,
             path=True, n=61, e4m3=False, lens=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8), (16, 16), (16, 4), (16, 2), (8, 1), (24, 8), (40, 8), (28, 4), (4, 4)]
PAGES = [16, 32, 64, 128, 256]


def draw(rng):
    op = rng.choice(["mask", "attn", "attn", "weigh", "weigh", "select", "keep"])
    lens = rng.randint(0, 10 ** 6)
    if op == "mask":
        return dict(op=op, B=_log(rng, 1, 256), n=_log(rng, 2, 256), ragged=rng.random() < 0.5, lens=lens)
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128])
    c = dict(op=op, Hkv=Hkv, page=rng.choice(PAGES), lens=lens)
    if op in ("attn", "weigh"):
        tree = op == "attn"
        B = _log(rng, 1, 64)
        n = _log(rng, 2, 160) if tree else rng.choice([1, 1, 2, 4, _log(rng, 5, 2048), _log(rng, 5, 2048)])
        L = max(n, min(_log(rng, 64, 65536), 402653184 // (B * Hkv * D)))
        n = max(1, min(n, 1073741824 // (B * Hq * L)))
        c.update(B=B, n=n, ragged=rng.random() < 0.5, Hq=Hq, D=D, L=L, e4m3=rng.random() < 0.5)
        if not tree:
            c.update(causal=rng.random() < 0.8, decay=rng.choice([1.0, 1.0, 0.97, 0.5]))
        return c
    B = _log(rng, 1, 128)
    L = max(40, min(_log(rng, 64, 262144), 16777216 // (B * Hkv)))
    keep = max(4, int(L * rng.uniform(0.05, 0.95)))
    c.update(B=B, L=L, keep=keep, first=rng.randint(0, keep // 4), recent=rng.randint(0, keep // 2))
    if op == "keep":
        L = max(40, min(L, 402653184 // (B * Hkv * D)))
        c.update(D=D, e4m3=rng.random() < 0.5, path=rng.random() < 0.4, L=L)
        if c["path"]:
            n = rng.randint(4, 40)
            c.update(n=n, keep=rng.randint(1, min(n, 12)), first=0, recent=0)
        else:
            keep = max(4, min(keep, L - 1))
            c.update(keep=keep, first=min(c["first"], keep // 4), recent=min(c["recent"], keep // 2))
    return c


def _lengths(c):
    """(new tokens, keys) of every sequence.  The longest sequence is the first."""
    r = random.Random(c["lens"])
    B, n = c["B"], c.get("n", 0)
    if c["op"] in ("mask", "attn", "weigh"):
        # ragged trees have some nodes; other ragged chunks are single tokens half the time
        one = c["op"] == "weigh"
        new = [n] + [((1 if one and r.random() < 0.5 else r.randint(1, n)) if c["ragged"] else n)
                     for _ in range(B - 1)]
    else:
        new = [n] * B
    if c["op"] == "mask":
        return new, new
    lo = min(128, c["L"])
    return new, [c["L"]] + [max(m, r.randint(lo, c["L"])) for m in new[1:]]


def _counts(c, keys):
    """How many tokens each sequence keeps."""
    r = random.Random(c["lens"] + 1)
    return [r.randint(1, c["keep"]) if c.get("path") else min(k, c["keep"]) for k in keys]


def _parents(new, r):
    """Trees of drafted tokens, one after the other: a node's parent is a recent earlier node, or none (-1)."""
    out = []
    for n in new:
        wide = r.randint(2, 12)
        out += [-1] + [max(-1, i - 1 - int(r.random() ** 2 * min(i + 1, wide))) for i in range(1, n)]
    return out


# ------------------------------------------------------------------ inputs --

def _quantise(x):
    """E4M3 codes (as float8 values) and scale bytes of rows x [..., D]."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, k = torch.frexp(amax)                                               # amax = m * 2^k, 0.5 <= m < 1
    e = torch.where(m <= 0.875, k - 9, k - 8)                              # 448 = 0.875 * 2^9
    e = torch.where(amax == 0, torch.full_like(e, E_MIN), e).clamp(E_MIN, E_MAX)
    codes = torch.ldexp(x, -e.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _value(codes, scale):
    """FP32 values that codes and scale bytes stand for."""
    return codes.float() * torch.ldexp(torch.ones((), device=codes.device), scale.int() - 127).unsqueeze(-1)


def _randn(shape, g, spread=False):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if spread:   # channels of unlike size, as keys have them
        x = x * torch.exp(0.7 * torch.randn(shape[-1], generator=g, device="cuda")).to(torch.bfloat16)
    return x


def _table(c, keys, g):
    """Block table with shuffled pages, and how many pages there are: some spare ones between the sequences'."""
    counts = [-(-k // c["page"]) for k in keys]
    total, spare = sum(counts), 3
    order = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor([sum(counts[:i]) for i in range(len(counts))], device="cuda")
    cols = torch.arange(max(counts), device="cuda")
    at = (start.unsqueeze(1) + cols).clamp(max=total + spare - 1)
    used = cols < torch.tensor(counts, device="cuda").unsqueeze(1)
    return torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous(), total + spare


def _pages(c, num, g, s, names):
    for name in names:
        pages = _randn((num, c["Hkv"], c["page"], c["D"]), g, spread=name == "k")
        scale = None
        if c["e4m3"]:
            flat = pages.view(-1, c["D"])
            codes = torch.empty(flat.shape, dtype=torch.float8_e4m3fn, device="cuda")
            scale = torch.empty(flat.shape[0], dtype=torch.uint8, device="cuda")
            for i in range(0, flat.shape[0], 1 << 20):
                codes[i:i + (1 << 20)], scale[i:i + (1 << 20)] = _quantise(flat[i:i + (1 << 20)])
            pages, scale = codes.view(pages.shape), scale.view(pages.shape[:-1])
        s[name + "_pages"], s[name + "_scale"] = pages, scale


def _sums(shape, g):
    """Sums of attention weights: most of them small, a few large, some alike."""
    x = torch.rand(shape, generator=g, device="cuda")
    return torch.where(x < 0.1, torch.round(x * 64) / 64, x ** 8 * 40)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, keys = _lengths(c)
    s = {"case": c, "max_q": max(new), "max_k": max(keys)}
    ragged = c.get("ragged", False)
    lead = (sum(new),) if ragged else (c["B"], c.get("n", 0))
    s["cu"] = _cu(new) if ragged else None
    if c["op"] == "mask":
        s["parents"] = _ints(_parents(new, random.Random(seed))).view(lead)
        return s
    s["block_table"], num = _table(c, keys, g)
    s["keys"] = _ints(keys)
    if c["op"] == "select":
        s["sums"] = _sums((num, c["Hkv"], c["page"]), g)
        return s
    _pages(c, num, g, s, ("k",) if c["op"] == "weigh" else ("k", "v"))
    if c["op"] == "attn":
        s["q"] = _randn(lead + (c["Hq"], c["D"]), g)
        parents = _ints(_parents(new, random.Random(c["lens"]))).view(lead)
        s["tree"] = _mask_plain({"case": c, "parents": parents, "cu": s["cu"], "max_q": s["max_q"]})["mask"]
    elif c["op"] == "weigh":
        s["q"] = _randn(lead + (c["Hq"], c["D"]), g)
        # older sums of the size of what this call adds
        s["sums"] = _sums((num, c["Hkv"], c["page"]), g) * (c["n"] * c["Hq"] / c["Hkv"] / c["L"] / 4)
        s["lse"] = _unpad(s, torch.logsumexp(_scores(s), -1).reshape(c["B"], c["Hq"], -1))
    else:
        s["sums"] = _sums((num, c["Hkv"], c["page"]), g)
        counts = _counts(c, keys)
        most = max(counts)
        i = torch.arange(most, device="cuda", dtype=torch.int32)
        s["counts"] = _ints(counts)
        behind = i >= s["counts"].unsqueeze(1)
        if c["path"]:       # the first drafted token and a path down from it
            past = [k - m for k, m in zip(keys, new)]
            r = random.Random(seed)
            rows = [sorted(r.sample(range(1, c["n"]), m - 1)) for m in counts]
            s["start"] = _ints(past)
            s["index"] = _ints([[p] + [p + x for x in row] + [-1] * (most - 1 - len(row))
                                for p, row in zip(past, rows)]).unsqueeze(1)
        else:               # some of the first and of the last tokens, and others from between them
            x = torch.rand((c["B"], c["Hkv"], max(keys)), generator=g, device="cuda")
            x = _protect(x, s["keys"], c["first"], c["recent"])
            s["start"] = None
            at = x.topk(most, dim=-1).indices.to(torch.int32)
            at = torch.where(behind.unsqueeze(1), torch.full_like(at, 2 ** 30), at).sort(-1).values
            s["index"] = torch.where(behind.unsqueeze(1), torch.full_like(at, -1), at).contiguous()
    return s


# ------------------------------------------------------------- plain forms --

def _padded(s, x):
    """Packed rows x as [B, max_q, ...], and the number of new tokens of each sequence."""
    c = s["case"]
    if s["cu"] is None:
        return x, torch.full((c["B"],), s["max_q"], device="cuda")
    row = torch.arange(s["max_q"], device="cuda")
    at = (s["cu"][:-1].long().unsqueeze(1) + row).clamp(max=x.shape[0] - 1)
    return x[at], (s["cu"][1:] - s["cu"][:-1]).long()


def _of_rows(s, total):
    """(sequence, token in it) of packed rows."""
    i = torch.arange(total, device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), i, right=True)
    return b, i - s["cu"][b]


def _unpad(s, x):
    """[B, Hq, max_q] as [Hq, total], where rows are packed."""
    if s["cu"] is None:
        return x.contiguous()
    b, r = _of_rows(s, s["q"].shape[0])
    return x[b, :, r].t().contiguous()


def _mask_plain(s):
    parents, new = _padded(s, s["parents"])
    B, n = parents.shape
    i = torch.arange(n, device="cuda")
    real = i < new.unsqueeze(1)
    # child to parent and to itself; its powers reach all ancestors
    a = (parents.unsqueeze(2) == i) | (i.unsqueeze(1) == i)
    a = (a & real.unsqueeze(2) & real.unsqueeze(1)).float()
    for _ in range(max(1, (n - 1).bit_length())):
        a = ((a @ a) > 0).float()
    words = -(-n // 32)
    bits = torch.nn.functional.pad(a, (0, 32 * words - n)).view(B, n, words, 32).long()
    mask = (bits << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32)
    depth = a.sum(-1).to(torch.int32) - 1
    if s["cu"] is None:
        return {"mask": mask, "depth": depth}
    b, r = _of_rows(s, s["parents"].shape[0])
    return {"mask": mask[b, r], "depth": depth[b, r]}


def _gather(s, name):
    """Keys or values [B, Hkv, keys, D] in FP32, padded to the longest sequence."""
    c = s["case"]
    table = s["block_table"].clamp(min=0).long()
    pages = s[name + "_pages"]
    if c["e4m3"]:
        x = _value(pages.view(torch.uint8)[table].view(torch.float8_e4m3fn), s[name + "_scale"][table])
    else:
        x = pages[table].float()
    return x.permute(0, 2, 1, 3, 4).reshape(c["B"], c["Hkv"], -1, c["D"])[:, :, :s["max_k"]]


def _scores(s):
    """Masked scores [B, Hkv, group, max_q, keys] in FP32: a tree's mask, the causal one, or the sequence's end."""
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    n, L, grp = s["max_q"], s["max_k"], Hq // Hkv
    q, new = _padded(s, s["q"])
    q = q.float().reshape(B, n, Hkv, grp, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, grp * n, D)
    x = (q @ _gather(s, "k").transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, grp, n, L)
    key = torch.arange(L, device="cuda")
    keys, row = s["keys"].long().view(B, 1, 1), torch.arange(n, device="cuda").view(1, n, 1)
    past = keys - new.view(B, 1, 1)
    if "tree" in s:
        tree = _padded(s, s["tree"])[0]
        j = (key - past).clamp(min=0, max=32 * tree.shape[-1] - 1)           # [B, 1, L]
        bit = (tree.long().gather(2, (j // 32).expand(B, n, L)) >> (j % 32)) & 1
        hidden = (key >= past) & ((bit == 0) | (key >= keys))
    else:
        hidden = key > (past + row if c["causal"] else (keys - 1).expand(B, n, 1))
    return x.masked_fill_(hidden.view(B, 1, 1, n, L), -math.inf)


def _attn_plain(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    n, L, grp = s["max_q"], s["max_k"], Hq // Hkv
    x = _scores(s)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, grp * n, L) @ _gather(s, "v")).view(B, Hkv, grp, n, D)
    o = (o / l.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(torch.bfloat16)
    lse = _unpad(s, (m + l.log()).view(B, Hq, n))
    if s["cu"] is None:
        return {"o": o, "lse": lse}
    return {"o": o[_of_rows(s, s["q"].shape[0])], "lse": lse}


def _weigh_plain(s):
    c = s["case"]
    B, Hq, Hkv, P = c["B"], c["Hq"], c["Hkv"], c["page"]
    n, L, grp = s["max_q"], s["max_k"], Hq // Hkv
    if s["cu"] is None:
        lse, new = s["lse"], torch.full((B,), n, device="cuda")
    else:       # rows behind a sequence's own give nothing
        lse, new = _padded(s, s["lse"].t())
        real = torch.arange(n, device="cuda") < new.unsqueeze(1)
        lse = lse.masked_fill(~real.unsqueeze(2), math.inf).transpose(1, 2)
    x = _scores(s)
    w = x.sub_(lse.reshape(B, Hkv, grp, n, 1)).exp_().sum((2, 3))                     # [B, Hkv, L]
    key = torch.arange(L, device="cuda")
    b, t = torch.nonzero(key < s["keys"].unsqueeze(1), as_tuple=True)                 # (sequence, token) of all keys
    page, slot = s["block_table"][b, t // P].long(), t % P
    old = s["sums"][page, :, slot]
    old = torch.where((t >= s["keys"][b] - new[b]).unsqueeze(1), torch.zeros_like(old), old)
    s["sums"][page, :, slot] = c["decay"] * old + w[b, :, t]
    return {"sums": s["sums"]}


def _protect(x, keys, first, recent):
    """Scores x [B, Hkv, L] with the first and the last tokens above all others, and nothing behind the last."""
    key = torch.arange(x.shape[-1], device="cuda")
    keys = keys.view(-1, 1, 1)
    x = x.masked_fill((key < first) | (key >= keys - recent), math.inf)
    return x.masked_fill(key >= keys, -math.inf)


def _select_plain(s):
    c = s["case"]
    P, keep = c["page"], min(c["keep"], s["max_k"])
    key = torch.arange(s["max_k"], device="cuda")
    x = s["sums"][s["block_table"].clamp(min=0).long()[:, key // P], :, key % P].transpose(1, 2)
    x = _protect(x, s["keys"], c["first"], c["recent"])
    # ties go to the lowest index: a stable sort
    at = x.sort(dim=-1, descending=True, stable=True).indices[..., :keep].to(torch.int32)
    kept = s["keys"].clamp(max=c["keep"])
    behind = torch.arange(keep, device="cuda") >= kept.view(-1, 1, 1)
    at = torch.where(behind, torch.full_like(at, 2 ** 30), at).sort(-1).values
    at = torch.where(behind, torch.full_like(at, -1), at)
    return {"index": torch.nn.functional.pad(at, (0, c["keep"] - keep), value=-1), "kept": kept}


def _keep_plain(s):
    c = s["case"]
    P, Hkv = c["page"], c["Hkv"]
    index = s["index"].expand(-1, Hkv, -1)
    b, h, i = torch.nonzero(index >= 0, as_tuple=True)
    table = s["block_table"]
    src, dst = index[b, h, i].long(), i if s["start"] is None else i + s["start"][b]
    of = table[b, src // P].long(), h, src % P
    to = table[b, dst // P].long(), h, dst % P
    out = {}
    for name in ("k_pages", "v_pages", "k_scale", "v_scale", "sums"):
        if s[name] is not None:
            x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
            x[to] = x[of]
            out[name] = s[name]
    return out


# --------------------------------------------------------------------- run --

def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"mask": _mask_plain, "attn": _attn_plain, "weigh": _weigh_plain, "select": _select_plain,
                "keep": _keep_plain}[c["op"]](s)
    import exact_attention_78_gb300 as fa

    if c["op"] == "mask":
        mask, depth = fa.tree_mask(s["parents"], cu_seqlens=s["cu"], max_q=s["max_q"])
        return {"mask": mask, "depth": depth}
    if c["op"] == "attn":
        o, lse = fa.fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["keys"], tree=s["tree"],
                              cu_seqlens=s["cu"], max_q=s["max_q"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"o": o, "lse": lse}
    if c["op"] == "weigh":
        fa.cache_weights(s["q"], s["lse"], s["k_pages"], s["sums"], s["block_table"], s["keys"], causal=c["causal"],
                         decay=c["decay"], cu_seqlens=s["cu"], max_q=s["max_q"], k_scale=s["k_scale"])
        return {"sums": s["sums"]}
    if c["op"] == "select":
        index, kept = fa.cache_select(s["sums"], s["block_table"], s["keys"], c["keep"], first=c["first"],
                                      recent=c["recent"])
        return {"index": index, "kept": kept}
    fa.cache_keep(s["k_pages"], s["v_pages"], s["block_table"], s["index"], s["counts"], start=s["start"],
                  k_scale=s["k_scale"], v_scale=s["v_scale"], sums=s["sums"])
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale", "sums") if s[x] is not None}


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    new, keys = _lengths(c)
    if c["op"] == "mask":
        words = -(-max(new) // 32)
        return {"bytes": 4 * sum(new) * (words + 2), "flops": sum(new) * words}
    Hkv = c["Hkv"]
    pages = 4 * sum(-(-k // c["page"]) for k in keys)
    if c["op"] == "select":
        return {"bytes": 4 * Hkv * (sum(keys) + sum(_counts(c, keys))) + pages, "flops": sum(keys) * Hkv}
    D = c["D"]
    held = (D + 1 if c["e4m3"] else 2 * D) * Hkv           # bytes of one token's keys in the cache
    if c["op"] == "keep":       # rows that stay where they are are not moved
        moved = sum(_counts(c, keys)) - c["B"] * (1 if c["path"] else c["first"])
        lists = 4 * (1 if c["path"] else Hkv) * sum(_counts(c, keys))
        return {"bytes": max(1, moved) * 2 * (2 * held + 4 * Hkv) + lists, "flops": 0}
    past = sum(n * (k - n) for n, k in zip(new, keys))
    if c["op"] == "attn":
        parents, depth, seen, first = _parents(new, random.Random(c["lens"])), [], past, 0
        for n in new:
            depth = []
            for p in parents[first:first + n]:
                depth.append(1 if p < 0 else depth[p] + 1)
            seen, first = seen + sum(depth), first + n
        words = -(-max(new) // 32)
        return {"bytes": 2 * sum(keys) * held + pages + sum(new) * (c["Hq"] * (4 * D + 4) + 4 * words),
                "flops": 4 * seen * c["Hq"] * D}
    seen = past + sum(n * (n + 1) // 2 if c["causal"] else n * n for n in new)
    return {"bytes": sum(keys) * (held + 8 * Hkv) - 4 * Hkv * sum(new) + pages + sum(new) * c["Hq"] * (2 * D + 4),
            "flops": 2 * seen * c["Hq"] * D}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The definitions in 64 bits, one sequence and head at a time."""
    c = case
    if c["op"] in ("mask", "select", "keep"):       # whole numbers, or rows moved as they are
        return None
    s = prepare(c, seed)
    new, keys = _lengths(c)
    if work(c)["flops"] > 2.5e12:
        return None
    D, P, grp = c["D"], c["page"], c["Hq"] // c["Hkv"]

    def rows(name, b):    # keys or values of sequence b, [L, Hkv, D] in 64 bits
        at = torch.arange(keys[b], device="cuda")
        page, slot = s["block_table"][b][at // P].long(), at % P
        if not c["e4m3"]:
            return s[name + "_pages"][page, :, slot].double()
        codes = s[name + "_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).double()
        return codes * torch.exp2(s[name + "_scale"][page, :, slot].double() - 127.0).unsqueeze(-1)

    trees = _parents(new, random.Random(c["lens"])) if c["op"] == "attn" else None
    sums = s["sums"].double() if c["op"] == "weigh" else None
    o_all, l_all, first = [], [], 0
    for b in range(c["B"]):
        n, L = new[b], keys[b]
        q = (s["q"][b] if s["cu"] is None else s["q"][first:first + n]).double()
        sees = torch.ones(n, L, dtype=torch.bool)
        if trees is not None:
            sees[:, L - n:] = False
            for i in range(n):
                j = i
                while j >= 0:
                    sees[i, L - n + j] = True
                    j = trees[first + j]
        elif c["causal"]:
            sees = sees.tril(L - n)
        sees = sees.cuda()
        k = rows("k", b)
        if trees is None:
            lse = s["lse"][b] if s["cu"] is None else s["lse"][:, first:first + n]
            at = torch.arange(L, device="cuda")
            page, slot = s["block_table"][b][at // P].long(), at % P
            old = sums[page, :, slot] * c["decay"]
            old[L - n:] = 0
            for h in range(c["Hq"]):
                x = (q[:, h] @ k[:, h // grp].T / math.sqrt(D)).masked_fill(~sees, -math.inf)
                old[:, h // grp] += torch.exp(x - lse[h].double().unsqueeze(-1)).sum(0)
            sums[page, :, slot] = old
            first += n
            continue
        v = rows("v", b)
        o = torch.empty(n, c["Hq"], D, dtype=torch.float64, device="cuda")
        lse = torch.empty(c["Hq"], n, dtype=torch.float64, device="cuda")
        for h in range(c["Hq"]):
            x = (q[:, h] @ k[:, h // grp].T / math.sqrt(D)).masked_fill(~sees, -math.inf)
            lse[h] = torch.logsumexp(x, -1)
            o[:, h] = torch.exp(x - lse[h].unsqueeze(-1)) @ v[:, h // grp]
        o_all.append(o)
        l_all.append(lse)
        first += n
    if trees is None:
        return {"sums": sums}
    if s["cu"] is None:
        return {"o": torch.stack(o_all), "lse": torch.stack(l_all)}
    return {"o": torch.cat(o_all), "lse": torch.cat(l_all, 1)}
