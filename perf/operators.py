"""Operators of a paged key/value cache: their cases, inputs, plain forms and exact values.

Four operators, in the order in which one serving step runs them:

  rope      rotary positions of q or k [B, H, N, D]: forward, or the gradient (the transposed rotation)
  append    rotate the new tokens' q and k, and write k and v into the pages of a cache
  attend    attention of ragged chunks of new tokens over the paged cache (one token per sequence: decode)
  weigh     add every cached key's attention weight over the call's rows to the cache's running sums
  evict     keep the heaviest and the most recent keys of every key/value head, moved into other pages

`rope` is also the training form of the rotation that `append` does.  `run` computes them with elementary
torch operations in fp32 (angles in 64 bits) where `own` is false, and through the package where it is true.

Layouts: q [T, H, D], k and v [T, H_kv, D], packed sequence after sequence (cu [B + 1]); cache pages
[pages, H_kv, page, D]; weights [pages, H_kv, page]; table [B, pages per sequence]; kv_len [B] counts a
sequence's cached keys, its new ones included.  New token i of n sees the keys below kv_len - n + i + 1.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the rotation of q in a training step at the long-sequence size of the benchmark's forward pass
        dict(name="rope fwd 1x16x16384x128", op="rope", B=1, H=16, N=16384, D=128, rot=128, type="bf16",
             interleaved=False, inverse=False, base=10000.0, factor=1.0, mscale=1.0),
        # its gradient for an encoder-shaped fp32 batch, half of each head rotated, adjacent pairs
        dict(name="rope bwd 32x8x512x64 f32", op="rope", B=32, H=8, N=512, D=64, rot=32, type="f32",
             interleaved=True, inverse=True, base=10000.0, factor=1.0, mscale=1.0),
        # one decode step of a small batch: a few KB, all latency
        dict(name="append decode 16", op="append", B=16, n=1, n_min=1, kv=2000, kv_min=37, H=32, Hkv=8, D=128,
             rot=128, page=16, type="bf16", interleaved=False, base=500000.0, factor=1.0, mscale=1.0),
        # ragged prompt chunks into a long cache, positions stretched by a factor for the long context
        dict(name="append chunks 6x1024", op="append", B=6, n=1024, n_min=700, kv=30000, kv_min=1024, H=32, Hkv=8,
             D=128, rot=64, page=64, type="bf16", interleaved=True, base=10000.0, factor=4.0, mscale=1.1386),
        # decode of one sequence in fp32: the repository's single-query size
        dict(name="attend decode 1x16384 f32", op="attend", B=1, n=1, n_min=1, kv=16384, kv_min=16384, H=8, Hkv=8,
             D=64, page=64, type="f32"),
        # decode of a ragged batch with grouped heads and small pages
        dict(name="attend decode 16x8191 gqa", op="attend", B=16, n=1, n_min=1, kv=8191, kv_min=500, H=32, Hkv=8,
             D=128, page=16, type="bf16"),
        # chunks of new tokens over long caches: few rows, many keys
        dict(name="attend chunks 3x250/16384", op="attend", B=3, n=250, n_min=97, kv=16384, kv_min=9001, H=32, Hkv=8,
             D=128, page=32, type="bf16"),
        # whole prompts
        dict(name="attend prompts 4x4096", op="attend", B=4, n=4096, n_min=3001, kv=4096, kv_min=3001, H=16, Hkv=16,
             D=128, page=128, type="bf16"),
        # the weights of a decode step
        dict(name="weigh decode 16x8191 gqa", op="weigh", B=16, n=1, n_min=1, kv=8191, kv_min=500, H=32, Hkv=8,
             D=128, page=16, type="bf16"),
        # the weights of prompt chunks
        dict(name="weigh chunks 4x1024/4096", op="weigh", B=4, n=1024, n_min=513, kv=4096, kv_min=2050, H=16, Hkv=4,
             D=64, page=64, type="bf16"),
        # one long sequence cut to a quarter
        dict(name="evict 1x16384 to 4096", op="evict", B=1, kv=16384, kv_min=16384, Hkv=8, D=128, page=64, keep=4096,
             recent=256, type="bf16"),
        # a ragged batch cut back, some sequences below the limit already
        dict(name="evict 16x6000 to 2048", op="evict", B=16, kv=6000, kv_min=1500, Hkv=8, D=128, page=16, keep=2048,
             recent=128, type="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "weigh", "evict"])
    kind = "f32" if rng.random() < 0.25 else "bf16"
    D = rng.choice([32, 64, 96, 128]) if kind == "f32" else rng.choice([64, 128])
    rot = 16 * rng.randint(1, D // 16)
    turn = dict(rot=rot, interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                factor=rng.choice([1.0, 1.0, 4.0, 8.0]), mscale=rng.choice([1.0, 1.0, 1.1386]))
    if op == "rope":
        B, H = _log(rng, 1, 16), rng.randint(1, 24)
        N = _log(rng, 1, max(1, (1 << 24) // (B * H * D)))
        return dict(op=op, B=B, H=H, N=N, D=D, type=kind, inverse=rng.random() < 0.5, **turn)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "evict":
        B = _log(rng, 1, 16)
        kv = _log(rng, 40, 60000 // B)
        keep = rng.randint(kv // 8 + 1, kv)
        return dict(op=op, B=B, kv=kv, kv_min=rng.randint(kv // 4 + 1, kv), Hkv=Hkv, D=D, page=page, keep=keep,
                    recent=rng.randint(0, keep), type=kind)
    B = _log(rng, 1, 12)
    kv = _log(rng, 16, min(20000, 60000 // B))
    n = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(kv, 3000 // B)))
    if kind == "f32" and op != "append":
        n = min(n, 64)
    n = max(1, min(n, 200_000_000_000 // (4 * D * B * kv * H)))
    kv_min = rng.randint(max(n, kv // 4), max(n, kv))
    sizes = dict(op=op, B=B, n=n, n_min=rng.randint(1, n), kv=max(n, kv), kv_min=kv_min, H=H, Hkv=Hkv, D=D, page=page,
                 type=kind)
    return {**sizes, **turn} if op == "append" else sizes


def _spread(lo, hi, count):
    """`count` lengths from hi down to lo, out of order."""
    return [hi - ((i * 5) % count) * (hi - lo) // max(1, count - 1) if count > 1 else hi for i in range(count)]


def _lens(c):
    kv = _spread(c["kv_min"], c["kv"], c["B"])
    n = _spread(c["n_min"], c["n"], c["B"]) if "n" in c else [0] * c["B"]
    return [min(a, b) for a, b in zip(n, kv)], kv


def work(c):
    es = 2 if c["type"] == "bf16" else 4
    if c["op"] == "rope":
        e = c["B"] * c["H"] * c["N"] * c["D"]
        return {"bytes": 2 * e * es + 4 * c["N"], "flops": 3 * c["B"] * c["H"] * c["N"] * c["rot"]}
    n, kv = _lens(c)
    T, L, D, Hkv = sum(n), sum(kv), c["D"], c["Hkv"]
    if c["op"] == "evict":
        kept = sum(min(x, c["keep"]) for x in kv) * Hkv
        return {"bytes": 4 * L * Hkv + 2 * kept * (2 * D * es + 4) + 4 * kept, "flops": L * Hkv}
    H = c["H"]
    if c["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * Hkv) * D * es + 4 * T * (Hkv + 1), "flops": 3 * T * (H + Hkv) * c["rot"]}
    seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(n, kv)) * H
    if c["op"] == "attend":
        return {"bytes": 2 * T * H * D * es + 4 * T * H + 2 * L * Hkv * D * es, "flops": 4 * D * seen}
    return {"bytes": T * H * D * es + 4 * T * H + L * Hkv * (D * es + 8), "flops": 2 * D * seen}


# ------------------------------------------------------------------ inputs

def _freq(c, dev):
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev)
    return c["base"] ** (-2.0 * i / c["rot"]) / c["factor"]


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    dt = TYPES[c["type"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=dev, dtype=torch.float32).to(dt)  # noqa: E731
    if c["op"] == "rope":
        c["x"] = normal(c["B"], c["H"], c["N"], c["D"])
        c["freq"] = _freq(c, dev)
        c["pos"] = torch.arange(c["N"], device=dev, dtype=torch.int32) + seed % 1000
        return c
    n, kv = _lens(c)
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    per = [-(-x // page) for x in kv]
    dst = [-(-min(x, c["keep"]) // page) for x in kv] if c["op"] == "evict" else [0] * B
    pages = sum(per) + sum(dst) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)

    def table(counts, at):  # unused entries name no page
        t = torch.full((B, max(counts)), -1, dtype=torch.int32)
        where = torch.zeros(B, max(counts), dtype=torch.bool)
        for b, m in enumerate(counts):
            where[b, :m] = True
        t, where = t.to(dev), where.to(dev)
        t[where] = order[at:at + sum(counts)]
        return t

    c["table"] = table(per, 0)
    c["k_cache"] = normal(pages, Hkv, page, D)
    c["v_cache"] = normal(pages, Hkv, page, D)
    # what a few hundred rows' attention leaves: most keys light, some heavy
    c["weights"] = torch.rand(pages, Hkv, page, generator=g, device=dev).pow_(4).mul_(3.0)
    c["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    c["max_kv"] = max(kv)
    if c["op"] == "evict":
        c["dst"] = table(dst, sum(per))
        c["spare"] = order[-1:].long()
        return c
    T = sum(n)
    c["max_q"] = max(n)
    c["cu"] = torch.tensor([0] + n, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)
    c["scale"] = 1.0 / math.sqrt(D)
    # the new tokens' q, k and v come out of one projection: rows of all heads
    row = normal(T, (c["H"] + 2 * Hkv) * D)
    q, k, v = row.split([c["H"] * D, Hkv * D, Hkv * D], dim=1)
    c["q"], c["k"], c["v"] = q.view(T, c["H"], D), k.view(T, Hkv, D), v.view(T, Hkv, D)
    if c["op"] == "append":
        c["freq"] = _freq(c, dev)
        b, i = _rows(c)
        # a cache that was cut back earlier: positions run ahead of the slots
        c["pos"] = (c["kv_len"][b] - (c["cu"][1:] - c["cu"][:-1])[b] + i + seed % 5000).to(torch.int32)
    if c["op"] == "weigh":
        c["lse"] = _attend(c)["lse"]
    return c


# -------------------------------------------------------------- plain forms

def _rows(s):
    """Sequence and place in it of every packed row."""
    t = torch.arange(s["k"].shape[0] if "k" in s else s["q"].shape[0], device=s["cu"].device)
    b = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    return b, t - s["cu"][b]


def _turn(x, angle, rot, interleaved, mscale, inverse):
    """Rotated x: the pairs (2i, 2i + 1), or (i, i + rot / 2), of the first rot values of a head."""
    cos, sin = (torch.cos(angle) * mscale).float(), (torch.sin(angle) * mscale).float()
    sin = -sin if inverse else sin
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _gather(s, pages, limit):
    """Cached rows in order of their slots, [B, H_kv, limit, ...] in fp32; zero where no key is."""
    x = pages[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)[:, :, :limit].float()
    here = torch.arange(limit, device=x.device)[None, :] < s["kv_len"][:, None]
    here = here[:, None, :] if x.dim() == 3 else here[:, None, :, None]
    return torch.where(here, x, torch.zeros((), device=x.device))


def _scores(s):
    """Padded scores [B, H_kv, rows, keys] of the chunks, the mask of what they see, and the padding's index."""
    B, Hkv, G, n = s["kv_len"].shape[0], s["Hkv"], s["H"] // s["Hkv"], s["max_q"]
    at = s["cu"][:-1, None].long() + torch.arange(n, device=s["cu"].device)
    q = s["q"][at.clamp(max=s["q"].shape[0] - 1)].float()                       # [B, n, H, D]
    q = q.view(B, n, Hkv, G, -1).transpose(1, 2).reshape(B, Hkv, n * G, -1)
    x = torch.matmul(q, _gather(s, s["k_cache"], s["max_kv"]).transpose(2, 3)) * s["scale"]
    count = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(n, device=s["cu"].device).repeat_interleave(G)             # row = token * G + head of the group
    edge = (s["kv_len"] - count)[:, None] + i[None, :] + 1
    edge = torch.where(i[None, :] < count[:, None], edge, torch.zeros_like(edge))
    seen = torch.arange(s["max_kv"], device=x.device)[None, None, :] < edge[:, :, None]
    return x, seen[:, None]


def _unpad(s, x):
    """[B, H_kv, n * G, ...] back to packed [T, H, ...]."""
    b, i = _rows(s)
    G = s["H"] // s["Hkv"]
    x = x.unflatten(2, (s["max_q"], G))[b, :, i]                                  # [T, H_kv, G, ...]
    return x.flatten(1, 2)


def _attend(s):
    x, seen = _scores(s)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gather(s, s["v_cache"], s["max_kv"])) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]
    return {"o": _unpad(s, o).to(s["q"].dtype), "lse": _unpad(s, lse)}


def _weigh(s):
    x, seen = _scores(s)
    B, Hkv, G, n = s["kv_len"].shape[0], s["Hkv"], s["H"] // s["Hkv"], s["max_q"]
    at = (s["cu"][:-1, None].long() + torch.arange(n, device=x.device)).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"][at].view(B, n, Hkv, G).transpose(1, 2).reshape(B, Hkv, n * G, 1)
    p = torch.exp(x - lse).masked_fill(~seen, 0.0).sum(2)                         # [B, H_kv, keys]
    slot = torch.arange(s["max_kv"], device=x.device)
    page = s["table"].clamp(min=0).long()[:, slot // s["page"]]                   # [B, keys]
    head = torch.arange(Hkv, device=x.device)[None, :, None]
    s["weights"].index_put_((page[:, None, :], head, (slot % s["page"])[None, None, :]), p, accumulate=True)
    return {"weights": s["weights"]}


def _append(s):
    b, i = _rows(s)
    slot = (s["kv_len"][b] - (s["cu"][1:] - s["cu"][:-1])[b] + i).long()
    page, off = s["table"][b, slot // s["page"]].long(), slot % s["page"]
    angle = (s["pos"].double()[:, None] * s["freq"])[:, None, :]
    turn = (s["rot"], s["interleaved"], s["mscale"], False)
    s["k_cache"][page, :, off] = _turn(s["k"], angle, *turn)
    s["v_cache"][page, :, off] = s["v"]
    s["weights"][page, :, off] = 0.0
    return {"q": _turn(s["q"], angle, *turn), "k": s["k_cache"], "v": s["v_cache"], "weights": s["weights"]}


def _evict(s):
    L, keep = s["max_kv"], s["keep"]
    slot = torch.arange(L, device=s["kv_len"].device)
    length = s["kv_len"].long()
    recent = length.clamp(max=min(s["recent"], keep))
    old = slot[None, :] < (length - recent)[:, None]                             # candidates, by weight
    w = _gather(s, s["weights"], L)
    w = torch.where(old[:, None] & ~torch.isnan(w), w, torch.full_like(w, -math.inf))
    rank = torch.sort(torch.sort(w, dim=2, descending=True, stable=True)[1], dim=2)[1]
    kept = (old[:, None] & (rank < (keep - recent)[:, None, None])) | (~old & (slot < length[:, None]))[:, None]
    new_len = length.clamp(max=keep)
    width = min(keep, L)
    at = torch.sort(torch.where(kept, slot, slot + L), dim=2)[0][:, :, :width]
    there = torch.arange(width, device=at.device)
    valid = (there[None, :] < new_len[:, None])[:, None]
    index = torch.where(valid, at, torch.full_like(at, -1))
    at = at.clamp(max=L - 1)
    head = torch.arange(s["Hkv"], device=at.device)[None, :, None]
    seq = torch.arange(length.shape[0], device=at.device)[:, None, None]
    src = s["table"].clamp(min=0).long()[seq, at // s["page"]]
    to = s["dst"].long()[:, None, :].expand(-1, s["Hkv"], -1)
    to = to[:, :, (there // s["page"]).clamp(max=to.shape[2] - 1)]
    # what is behind a sequence's last kept key stays as it was: those rows go to a page that no sequence has
    to = torch.where(valid, to, s["spare"])
    off = (there % s["page"])[None, None, :]
    for pages in (s["k_cache"], s["v_cache"], s["weights"]):
        before = pages[s["spare"]]
        pages[to, head, off] = pages[src, head, at % s["page"]]
        pages[s["spare"]] = before
    full = torch.full(index.shape[:2] + (keep,), -1, dtype=torch.int32, device=index.device)
    full[:, :, :width] = index.to(torch.int32)
    return {"k": s["k_cache"], "v": s["v_cache"], "weights": s["weights"], "kept": full,
            "kv_len": new_len.to(torch.int32)}


def run(s):
    if s["op"] == "rope":
        if own:
            import exact_memory_efficient_b200 as m
            return m.rope(s["x"], s["pos"], s["freq"], interleaved=s["interleaved"], mscale=s["mscale"],
                          inverse=s["inverse"])
        angle = s["pos"].double()[:, None] * s["freq"]
        return _turn(s["x"], angle, s["rot"], s["interleaved"], s["mscale"], s["inverse"])
    if not own:
        return {"append": _append, "attend": _attend, "weigh": _weigh, "evict": _evict}[s["op"]](s)
    import exact_memory_efficient_b200 as m
    if s["op"] == "append":
        q = m.paged_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["weights"], s["cu"], s["kv_len"],
                           s["table"], s["pos"], s["freq"], interleaved=s["interleaved"], mscale=s["mscale"])
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"], "weights": s["weights"]}
    if s["op"] == "attend":
        o, lse = m.attention_paged(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_len"], s["table"], s["max_q"],
                                   s["max_kv"], s["scale"])
        return {"o": o, "lse": lse}
    if s["op"] == "weigh":
        m.attention_paged_weights(s["q"], s["lse"], s["k_cache"], s["weights"], s["cu"], s["kv_len"], s["table"],
                                  s["max_q"], s["max_kv"], s["scale"])
        return {"weights": s["weights"]}
    kept, kv_len = m.paged_evict(s["k_cache"], s["v_cache"], s["weights"], s["table"], s["kv_len"], s["dst"],
                                 s["keep"], s["recent"])
    return {"k": s["k_cache"], "v": s["v_cache"], "weights": s["weights"], "kept": kept, "kv_len": kv_len}


# ------------------------------------------------------------- exact values

def _complex_turn(x, pos, c, sign):
    """The rotation as a product of complex numbers, in 64 bits; x [..., rows, D], pos [rows]."""
    half, rot = c["rot"] // 2, c["rot"]
    x = x.double()
    pairs = x[..., :rot].unflatten(-1, (half, 2)) if c["interleaved"] else x[..., :rot].unflatten(-1, (2, half)).mT
    z = torch.view_as_complex(pairs.contiguous())
    freq = 1.0 / (c["factor"] * c["base"] ** (torch.arange(half, dtype=torch.float64, device=x.device) / half))
    z = z * torch.polar(torch.full((), c["mscale"], dtype=torch.float64, device=x.device).expand(len(pos), half),
                        sign * pos.double()[:, None] * freq)
    pairs = torch.view_as_real(z)
    return torch.cat(((pairs if c["interleaved"] else pairs.mT).flatten(-2), x[..., rot:]), -1)


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence (and head by head where a whole one would not fit)."""
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _complex_turn(s["x"], s["pos"], s, -1.0 if s["inverse"] else 1.0)
    counts, lens, page = _lens(s)[0], _lens(s)[1], s["page"]
    G, cu = (s["H"] // s["Hkv"] if "H" in s else 0), s["cu"].tolist() if "cu" in s else None
    slots = [s["table"][b, :-(-x // page)].long().repeat_interleave(page)[:x] for b, x in enumerate(lens)]
    offs = [torch.arange(x, device="cuda") % page for x in lens]
    if s["op"] == "append":
        out = {"q": _complex_turn(s["q"].transpose(0, 1), s["pos"], s, 1.0).transpose(0, 1),
               "k": s["k_cache"].double(), "v": s["v_cache"].double(), "weights": s["weights"].double()}
        k = _complex_turn(s["k"].transpose(0, 1), s["pos"], s, 1.0).transpose(0, 1)
        for b, (n, x) in enumerate(zip(counts, lens)):
            p, o = slots[b][x - n:], offs[b][x - n:]
            out["k"][p, :, o] = k[cu[b]:cu[b + 1]]
            out["v"][p, :, o] = s["v"][cu[b]:cu[b + 1]].double()
            out["weights"][p, :, o] = 0.0
        return out
    if s["op"] == "evict":
        out = {k: s[f"{k}_cache" if k in "kv" else k].clone() for k in ("k", "v", "weights")}
        out["kept"] = torch.full((len(lens), s["Hkv"], s["keep"]), -1, dtype=torch.int32, device="cuda")
        out["kv_len"] = torch.tensor([min(x, s["keep"]) for x in lens], dtype=torch.int32, device="cuda")
        for b, x in enumerate(lens):
            recent = min(s["recent"], x)
            heavy = min(s["keep"], x) - recent
            for h in range(s["Hkv"]):
                w = s["weights"][slots[b], h, offs[b]][:x - recent].cpu().tolist()
                best = sorted(sorted(range(x - recent), key=lambda j: (-w[j], j))[:heavy]) + list(range(x - recent, x))
                kept = torch.tensor(best, device="cuda", dtype=torch.long)
                there = torch.arange(len(best), device="cuda")
                to = s["dst"][b, there // page].long()
                for name, pages in (("k", s["k_cache"]), ("v", s["v_cache"]), ("weights", s["weights"])):
                    out[name][to, h, there % page] = pages[slots[b][kept], h, offs[b][kept]]
                out["kept"][b, h, :len(best)] = kept.to(torch.int32)
        return {k: v.double() if v.is_floating_point() else v for k, v in out.items()}
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double()
    for b, (n, x) in enumerate(zip(counts, lens)):
        rows = slice(cu[b], cu[b + 1])
        hidden = torch.arange(x, device="cuda")[None, :] > torch.arange(x - n, x, device="cuda")[:, None]
        for h in range(s["H"]):
            k = s["k_cache"][slots[b], h // G, offs[b]].double()
            z = (s["q"][rows, h].double() @ k.T * s["scale"]).masked_fill_(hidden, -math.inf)
            if s["op"] == "weigh":
                # the rows' log-sums are an input here
                weights[slots[b], h // G, offs[b]] += (z - s["lse"][rows, h].double()[:, None]).exp_().sum(0)
                continue
            lse[rows, h] = torch.logsumexp(z, 1)
            o[rows, h] = torch.softmax(z, 1) @ s["v_cache"][slots[b], h // G, offs[b]].double()
    return {"weights": weights} if s["op"] == "weigh" else {"o": o, "lse": lse}
