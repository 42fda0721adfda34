"""Cases of the operators around a cache that is held to a budget: the rotation of tokens
that have several positions, one new token's attention that also adds up what weight
each cached tile got, and the eviction of the tiles with the least of it.

  axes    the fused projection's q, k, v rows to per-head normalised fp16 rows, rotated by
          positions along several axes (time, height, width of images and video)
  weigh   attention of one new token a sequence over the packed cache and the workspace,
          with its log-sum-exp and each tile's accumulated attention weight
  evict   every kv-head's tiles of least weight leave the cache; the others are moved
          together, so that the blocks at the end of a sequence's table are free

Heads are 64 query heads over 8 kv-heads, and 40 over 8, or smaller groups; lengths are
those of the decode, long-context and ragged serving workloads.
"""
import math

import torch

own = False

D = 128
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
# bits of a key and a value code, and whether the metadata is the lean kind
PRESETS = {"k4v2": (4, 2, False), "k4v4": (4, 4, False), "k2v2": (2, 2, False), "k4v2l": (4, 2, True)}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence behind a video: the latency of a decode step's rotation
        dict(name="axes decode 1", op="axes", n=1, hq=64, hkv=8, dtype="fp16", norm=True, sections="16-24-24", mixed=False,
             interleaved=False, rows=1, cols=1, start=5000),
        # one image of odd sides in bf16, its axes dealt to the pairs in turn
        dict(name="axes image 37x29", op="axes", n=37 * 29, hq=40, hkv=8, dtype="bf16", norm=True, sections="24-20-20",
             mixed=True, interleaved=False, rows=37, cols=29, start=211),
        # two axes, neighbouring pairs, fp32 rows of an encoder
        dict(name="axes 2d 4099 fp32", op="axes", n=4099, hq=16, hkv=16, dtype="fp32", norm=False, sections="16-16",
             mixed=False, interleaved=True, rows=64, cols=65, start=0),
        # a batch of video prompts out of the fused projection
        dict(name="axes video 65536", op="axes", n=65536, hq=64, hkv=8, dtype="bf16", norm=True, sections="16-24-24",
             mixed=False, interleaved=False, rows=32, cols=32, start=64),
        # one short conversation: latency
        dict(name="weigh 1x1000", op="weigh", preset="k4v2", hq=64, hkv=8, seqs=1, lo=1000, hi=1000, decay=1.0),
        # the decode batch
        dict(name="weigh 64x16384", op="weigh", preset="k4v2", hq=64, hkv=8, seqs=64, lo=16384, hi=16384, decay=1.0),
        # few long sequences, 2-bit keys: the context split over the GPU; weights that fade
        dict(name="weigh 4x131072 k2v2", op="weigh", preset="k2v2", hq=64, hkv=8, seqs=4, lo=131072, hi=131072, decay=0.99),
        # a ragged serving batch, 4-bit values, groups of five heads
        dict(name="weigh ragged k4v4", op="weigh", preset="k4v4", hq=40, hkv=8, seqs=37, lo=1024, hi=32768, decay=0.9),
        # one short conversation down to two thirds: latency
        dict(name="evict 1x3000", op="evict", preset="k4v2", hkv=8, seqs=1, lo=3000, hi=3000, part=0.66, first=1, last=2),
        # a serving batch at its budget: each sequence has one tile more than it may keep
        dict(name="evict 256 by one", op="evict", preset="k4v2", hkv=8, seqs=256, lo=1024, hi=32768, part=1.0, first=1,
             last=2),
        # a prefill batch down to half
        dict(name="evict 16x16384 half", op="evict", preset="k4v2", hkv=8, seqs=16, lo=16384, hi=16384, part=0.5, first=1,
             last=4),
        # few long sequences down to a quarter
        dict(name="evict 4x131072 quarter", op="evict", preset="k4v4", hkv=8, seqs=4, lo=131072, hi=131072, part=0.25,
             first=4, last=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "weigh", "weigh", "evict", "evict"])
    hq, hkv = rng.choice([(64, 8), (40, 8), (32, 8), (28, 4), (8, 1), (6, 2), (8, 8)])
    preset = rng.choice(sorted(PRESETS))
    if op == "axes":
        dtype = rng.choice(sorted(DTYPES))
        sections = rng.choice(["16-24-24", "24-20-20", "32-32", "16-16", "8-12-12", "64", "10-18-20-16", "4-2-2", "2-3-3"])
        return dict(op=op, n=_log(rng, 1, 65536 if dtype != "fp32" else 30000), hq=hq, hkv=hkv, dtype=dtype,
                    norm=rng.random() < 0.7, sections=sections, mixed=rng.random() < 0.5, interleaved=rng.random() < 0.4,
                    rows=_log(rng, 1, 200), cols=_log(rng, 1, 200), start=_log(rng, 1, 1000000) - 1)
    if op == "weigh":
        hi = _log(rng, 1, 131072)
        lo = max(0, hi - rng.choice([0, 1, hi // 3, hi - 1, hi]))
        return dict(op=op, preset=preset, hq=hq, hkv=hkv, seqs=_log(rng, 1, max(1, min(256, (1 << 20) // (hi + 64)))), lo=lo,
                    hi=hi, decay=rng.choice([1.0, 1.0, rng.uniform(0.5, 1.0)]))
    hi = _log(rng, 100, 131072)
    return dict(op=op, preset=preset, hkv=hkv, seqs=_log(rng, 1, max(1, min(256, 524288 // hi))), lo=rng.choice([0, hi // 3, hi]),
                hi=hi, part=rng.choice([1.0, 0.5, rng.uniform(0.0, 1.0)]), first=rng.choice([0, 1, 4]),
                last=rng.choice([0, 1, 2, 16]))


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], spread over its logarithm where it is wide; the case alone fixes them."""
    u = [(0.5 + 0.6180339887498949 * i) % 1.0 for i in range(n)]
    if hi > 10 * max(lo, 1):
        return [min(hi, max(lo, int(round(max(lo, 1) * math.exp(x * math.log(hi / max(lo, 1))))))) for x in u]
    return [lo + int(x * (hi - lo + 1)) if hi > lo else lo for x in u]


def _record_bytes(preset):
    kb, vb, lean = PRESETS[preset]
    return D * D * (kb + vb) // 8 + (1536 if lean else 2048)


def _axes(case):
    """The axis of each rotated pair: the axes' sections one after the other, or dealt in turn while a section lasts."""
    left = [int(x) for x in case["sections"].split("-")]
    if not case["mixed"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _budgets(case, lens):
    """Tiles that each sequence may keep: a part of its whole ones, or (part 1) all but one."""
    return [max(0, n // D - 1) if case["part"] == 1.0 else int(n // D * case["part"]) for n in lens]


# ------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(g, preset, blocks, hkv):
    """Packed records: uniform codes, and the metadata that normalised tiles have: row and
    column scales about 1, zeros about three standard deviations below, steps to match."""
    kb, vb, lean = PRESETS[preset]
    codes = D * D * (kb + vb) // 8
    rec = torch.empty(blocks, hkv, _record_bytes(preset), dtype=torch.uint8, device="cuda")
    rec[..., :codes] = torch.randint(0, 256, (blocks, hkv, codes), generator=g, device="cuda", dtype=torch.uint8)
    vecs = []
    for bits, value in ((kb, False), (vb, True)):
        r, c = (torch.exp(0.3 * _normal(g, blocks, hkv, D)) for _ in range(2))
        z = -3.0 * (1 + 0.1 * _normal(g, blocks, hkv, D).clamp(-3, 3))
        s = -2 * z / (2 ** bits - 1) * (1 + 0.1 * _normal(g, blocks, hkv, D).clamp(-3, 3))
        if lean:  # the scale that is constant in a group is part of its step and zero
            one = c if value else r
            vecs += [(r if value else c), s * one, z * one]
        else:
            vecs += [r, c, s, z]
    rec[..., codes:] = torch.stack(vecs, 2).half().reshape(blocks, hkv, -1).view(torch.uint8)
    return rec


def _paged(case, g, lens, tail):
    """Cache and block tables over a random permutation of its blocks: entries for the whole tiles and,
    with `tail`, for the partial one; those behind are -1."""
    used = [-(-n // D) if tail else n // D for n in lens]
    width = max(1, max(-(-n // D) for n in lens) + 1)
    blocks = sum(used) + 3
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    tables[torch.arange(width, device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]] = perm[: sum(used)]
    return dict(cache=_cache(g, case["preset"], blocks, case["hkv"]), tables=tables, width=width, blocks=blocks,
                lens=_i32(lens))


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "blocks": 1, "width": 1}
    op = case["op"]
    if op == "axes":
        n, hq, hkv, t = case["n"], case["hq"], case["hkv"], DTYPES[case["dtype"]]
        qkv = _normal(g, n, (hq + 2 * hkv) * D).mul_(1.7).to(t)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
        s["q_w"], s["k_w"] = ((1 + 0.2 * _normal(g, D)).to(t) if case["norm"] else None for _ in range(2))
        s["axes"] = _axes(case)
        half, axes = len(s["axes"]), max(s["axes"]) + 1
        s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        i = torch.arange(n, device="cuda")
        grid = (i // (case["rows"] * case["cols"]), i // case["cols"] % case["rows"], i % case["cols"], i % 7)
        s["pos"] = case["start"] + torch.stack(grid[:axes]).to(torch.int32)
        s["out"] = [torch.empty(n, h, D, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
    elif op == "weigh":
        lens, hq, hkv = _spread(case["seqs"], case["lo"], case["hi"]), case["hq"], case["hkv"]
        n = len(lens)
        s |= _paged(case, g, lens, False)
        s["max_len"] = max(lens)
        s["ws"] = (_normal(g, n, hkv, 2, D, D) * torch.exp(0.4 * _normal(g, n, hkv, 2, 1, D))).half()
        s["q"] = _normal(g, n, hq, D).half()
        # what earlier steps have left: a few steps' weight, heavier on some tiles
        s["weights"] = torch.exp(1.5 * _normal(g, n, hkv, s["width"])) * 0.02
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, hq, device="cuda")
    else:
        lens, hkv = _spread(case["seqs"], case["lo"], case["hi"]), case["hkv"]
        s |= _paged(case, g, lens, True)
        s["budgets"] = _i32(_budgets(case, lens))
        w = torch.exp(2 * _normal(g, len(lens), hkv, s["width"]))
        w[..., 0] *= 1000  # the first tile takes most of the weight
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.1] = 0.0  # and some tiles none
        at = torch.arange(s["width"], device="cuda")
        s["weights"] = w * (at < (s["lens"][:, None, None] + D - 1) // D)
        s["weights_out"] = torch.empty_like(s["weights"])
        s["lens_out"] = torch.empty_like(s["lens"])
        s["kept"] = torch.empty(w.shape, dtype=torch.int32, device="cuda")
    if own:
        import kv_cache_quantization_x128_gb300 as kv

        s["meta"] = kv.make_meta(case["hkv"], case.get("hq", case["hkv"]), s["blocks"], s["width"],
                                 preset=case.get("preset", "k4v2"))
        if op == "weigh":
            s["scratch"] = torch.empty(kv.decode_weights_scratch_bytes(s["meta"], case["seqs"]), dtype=torch.uint8,
                                       device="cuda")
    return s


# ------------------------------------------------------------------------ the passes
def run(s):
    op = s["case"]["op"]
    if own:
        return {"axes": _own_axes, "weigh": _own_weigh, "evict": _own_evict}[op](s)
    return {"axes": _axes_rope, "weigh": _weigh, "evict": _evict}[op](s)


def _own_axes(s):
    import kv_cache_quantization_x128_gb300 as kv

    c = s["case"]
    kv.kvarn_qk_norm_rope_axes(s["q"], s["k"], s["v"], s["pos"], s["axes"], *s["out"], s["meta"], q_weight=s["q_w"],
                               k_weight=s["k_w"], norm_eps=1e-6, inv_freq=s["inv_freq"], interleaved=c["interleaved"])
    return s["out"]


def _own_weigh(s):
    import kv_cache_quantization_x128_gb300 as kv

    kv.kvarn_decode_attention_weights(s["q"], s["cache"], s["ws"], s["tables"], s["lens"], s["weights"], s["out"],
                                      s["scratch"], s["meta"], decay=s["case"]["decay"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"], "weights": s["weights"]}


def _own_evict(s):
    import kv_cache_quantization_x128_gb300 as kv

    c = s["case"]
    kv.kvarn_evict_tiles(s["weights"], s["weights_out"], s["lens"], s["lens_out"], s["tables"], s["budgets"], s["kept"],
                         s["cache"], s["meta"], keep_first=c["first"], keep_last=c["last"])
    return {"kept": s["kept"], "lengths": s["lens_out"], "weights": s["weights_out"], "cache": s["cache"]}


def _axes_rope(s):
    c = s["case"]
    half = len(s["axes"])
    rot = 2 * half
    angle = s["pos"][s["axes"]].double().T * s["inv_freq"].double()
    cos, sin = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))

    def one(x, w, out):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        y = x.clone()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :half], x[..., half:rot])
        ya, yb = a * cos - b * sin, b * cos + a * sin
        y[..., :rot] = torch.stack((ya, yb), -1).flatten(-2) if c["interleaved"] else torch.cat((ya, yb), -1)
        out.copy_(y)

    one(s["q"], s["q_w"], s["out"][0])
    one(s["k"], s["k_w"], s["out"][1])
    s["out"][2].copy_(s["v"])
    return s["out"]


def _places(preset):
    """[channel, token]: the byte of a record and the shift in it of each key and each value code."""
    kb, vb, _ = PRESETS[preset]
    i, t = torch.arange(D, device="cuda")[:, None], torch.arange(D, device="cuda")[None]

    def nibbles(a, b):  # row b of 64 bytes, element a of it
        p = 4 * (a >> 3 & 1) + 2 * (a & 1) + (a >> 4 & 1)
        return 64 * b + 16 * (a >> 1 & 3) + 4 * (a >> 5) + (p >> 1), 4 * (p & 1)

    if kb == 4:
        k = nibbles(i, t)
    else:
        p = 4 * (i >> 4 & 3) + 2 * (i & 1) + (i >> 3 & 1)
        k = 32 * t + 8 * (i >> 1 & 3) + 4 * (i >> 6) + (p >> 2), 2 * (p & 3)
    if vb == 4:
        v = nibbles(t, i)
    else:
        p = 4 * (t >> 4 & 3) + 2 * (t & 1) + (t >> 3 & 1)
        v = (512 * (i >> 4) + 16 * (4 * (i & 7) + (t >> 1 & 3)) + 8 * (i >> 3 & 1) + 4 * (t >> 6) + (p >> 2), 2 * (p & 3))
    return k, (v[0] + D * D * kb // 8, v[1])


def _hadamard():
    i = torch.arange(D, device="cuda")
    x = i[:, None] & i[None]
    bits = sum((x >> b) & 1 for b in (0, 1, 2, 3, 4, 5, 6))
    return (1 - 2 * (bits & 1)).float() / math.sqrt(D)


def _dequant(rec, preset):
    """Records [..., bytes] -> K and V tiles [..., token, channel] in 32 bits, rotation undone."""
    kb, vb, lean = PRESETS[preset]
    codes = D * D * (kb + vb) // 8
    m = rec[..., codes:].contiguous().view(torch.float16).float().unflatten(-1, (-1, D))
    h = _hadamard()

    def one(place, bits, r, c, s, z):
        byte, shift = (x.expand(D, D).reshape(-1) for x in place)
        x = (rec[..., byte] >> shift.to(torch.uint8)) & (2 ** bits - 1)
        x = x.unflatten(-1, (D, D)).float()
        return ((x * s + z) * r * c).mT @ h

    pk, pv = _places(preset)
    row, col = (lambda x: x[..., :, None]), (lambda x: x[..., None, :])
    if lean:
        k = one(pk, kb, 1.0, col(m[..., 0, :]), row(m[..., 1, :]), row(m[..., 2, :]))
        v = one(pv, vb, row(m[..., 3, :]), 1.0, col(m[..., 4, :]), col(m[..., 5, :]))
    else:
        k = one(pk, kb, row(m[..., 0, :]), col(m[..., 1, :]), row(m[..., 2, :]), row(m[..., 3, :]))
        v = one(pv, vb, row(m[..., 4, :]), col(m[..., 5, :]), col(m[..., 6, :]), col(m[..., 7, :]))
    return k, v


def _cached(s):
    """K and V [sequence, kv-head, token, channel] of every cached token, in 32 bits, padded to the longest sequence."""
    lens, ws = s["lens"].long(), s["ws"]
    n, hkv = ws.shape[0], ws.shape[1]
    tiles = max(1, -(-s["max_len"] // D))
    k, v = _dequant(s["cache"][s["tables"][:, :tiles].long().clamp(min=0)], s["case"]["preset"])
    pos = torch.arange(tiles * D, device="cuda")
    tail = (pos[None] >= (lens // D * D)[:, None])[:, None, :, None]  # tokens of the partial tile are the workspace's

    def join(x, w):
        x = x.transpose(1, 2).reshape(n, hkv, tiles * D, D)
        return torch.where(tail, w.float().repeat(1, 1, tiles, 1), x)

    return join(k, ws[:, :, 0]), join(v, ws[:, :, 1]), pos


def _weigh(s):
    c = s["case"]
    hq, hkv, n = c["hq"], c["hkv"], c["seqs"]
    lens = s["lens"].long()
    k, v, at = _cached(s)
    tiles = at.numel() // D
    x = s["q"].float().reshape(n, hkv, hq // hkv, D) @ k.mT / math.sqrt(D)
    x = x.masked_fill((at[None] >= lens[:, None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    safe = top.clamp(min=-1e30)  # a sequence without tokens has no largest score
    p = torch.exp(x - safe)
    total = p.sum(-1, keepdim=True)
    p = p / total.clamp(min=1e-30)
    s["out"].copy_((p @ v).reshape(n, hq, D))
    s["lse"].copy_((safe + torch.log(total)).reshape(n, hq))
    got = p.unflatten(-1, (tiles, D)).sum(-1).sum(2)
    w = s["weights"][..., :tiles]
    there = (torch.arange(tiles, device="cuda") * D < lens[:, None])[:, None]
    w.copy_(torch.where(there, c["decay"] * w + got, w))
    return {"out": s["out"], "lse": s["lse"], "weights": s["weights"]}


def _evict(s):
    c, w, cache, tables = s["case"], s["weights"], s["cache"], s["tables"].long()
    width = w.shape[2]
    i = torch.arange(width, device="cuda").expand(w.shape)
    lens = s["lens"].long()[:, None, None]
    n = (lens // D).clamp(max=width)
    b = torch.minimum(n, s["budgets"].long()[:, None, None])
    first = b.clamp(max=c["first"])
    last = (b - first).clamp(max=c["last"])
    middle = (i >= first) & (i < n - last)
    best = torch.where(middle, w, -math.inf).argsort(dim=-1, descending=True, stable=True)
    rank = torch.empty_like(best).scatter_(-1, best, i.contiguous())
    chosen = middle & (rank < b - first - last)
    gone = middle & ~chosen
    moved = chosen & (i >= b - last)
    holes = gone & (i < b - last)
    listed_gone = (~gone).to(torch.int8).argsort(dim=-1, stable=True)
    listed_moved = (~moved).to(torch.int8).argsort(dim=-1, stable=True)
    kept = torch.where(holes, listed_moved.gather(-1, (holes.cumsum(-1) - 1).clamp(min=0)), i)
    kept = torch.where((i >= b - last) & (i < b), n - b + i, kept)
    kept = torch.where((i >= b) & (i < n), listed_gone.gather(-1, (i - b).clamp(min=0)), kept)
    kept = torch.where(i < n, kept, -1)
    s["kept"].copy_(kept)
    s["lens_out"].copy_(s["lens"] - ((n - b) * D)[:, 0, 0])
    src = torch.where(i == b, n.clamp(max=width - 1), kept.clamp(min=0))  # the partial tile's weight follows the last kept
    s["weights_out"].copy_(torch.where((i < b) | ((i == b) & (n < width)), w.gather(-1, src), 0.0))
    seq, head, to = torch.nonzero((i < b) & (kept != i), as_tuple=True)
    cache[tables[seq, to], head] = cache[tables[seq, kept[seq, head, to]], head]
    return {"kept": s["kept"], "lengths": s["lens_out"], "weights": s["weights_out"], "cache": cache}


# ------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "axes":
        n, heads = case["n"], case["hq"] + 2 * case["hkv"]
        size = DTYPES[case["dtype"]].itemsize
        return {"bytes": n * heads * D * (size + 2) + 4 * n * len(case["sections"].split("-")),
                "flops": n * (heads - case["hkv"]) * D * 8}
    rec, hkv = _record_bytes(case["preset"]), case["hkv"]
    lens = _spread(case["seqs"], case["lo"], case["hi"])
    if op == "weigh":
        hq = case["hq"]
        total = sum(n // D * hkv * rec + n % D * hkv * D * 4 + -(-n // D) * (hkv * 8 + 4) for n in lens)
        return {"bytes": total + len(lens) * hq * (D * 4 + 4), "flops": 4 * D * hq * sum(lens)}
    total = 0.0
    for n, budget in zip(lens, _budgets(case, lens)):
        t = n // D
        b = min(t, budget)
        first = min(case["first"], b)
        last = min(case["last"], b - first)
        middle, quota = t - first - last, b - first - last
        # evicted tiles below the last kept ones' places, for weights without an order, and the last kept ones
        moved = quota * (middle - quota) / max(1, middle) + (last if t > b else 0)
        total += hkv * (2 * rec * moved + t * (4 + 4 + 4)) + 4 * t + 12
    return {"bytes": total, "flops": 0}


# ------------------------------------------------------------------------ the definitions in 64 bits
def _tile64(rec, preset):
    """One (block, kv-head) batch of records [m, bytes] -> K, V [m, token, channel], float64."""
    kb, vb, lean = PRESETS[preset]
    m = rec.shape[0]
    nk, nv = D * D * kb // 8, D * D * vb // 8
    kc, vc = rec[:, :nk].long(), rec[:, nk:nk + nv].long()
    meta = rec[:, nk + nv:].contiguous().view(torch.float16).double().reshape(m, -1, D)

    def fours(b):  # [m, row, group(bits 1, 2), word(bits 5, 6), byte] -> [m, row, element]
        b = b.reshape(m, D, 4, 4, 4)
        e = torch.stack((b & 15, b >> 4), -1)                      # ..., byte (bit 3, bit 0), bit 4
        e = e.reshape(m, D, 4, 4, 2, 2, 2)                         # group, word, bit 3, bit 0, bit 4
        return e.permute(0, 1, 3, 6, 4, 2, 5).reshape(m, D, D)     # word, bit 4, bit 3, group, bit 0

    if kb == 4:
        k = fours(kc)
    else:
        b = kc.reshape(m, D, 4, 2, 4)                              # token, group, word, byte
        e = torch.stack([(b >> (2 * q)) & 3 for q in range(4)], -1).reshape(m, D, 4, 2, 4, 2, 2)
        # byte = bits 4, 5; crumb in it = bit 0, bit 3
        k = e.permute(0, 1, 3, 4, 6, 2, 5).reshape(m, D, D)
    if vb == 4:
        v = fours(vc).mT
    else:
        b = vc.reshape(m, 8, 8, 4, 2, 2, 4)                        # panel, i & 7, group, bit 3 of i, word, byte
        e = torch.stack([(b >> (2 * q)) & 3 for q in range(4)], -1).reshape(m, 8, 8, 4, 2, 2, 4, 2, 2)
        # byte = bits 4, 5 of t; crumb = bit 0, bit 3 of t
        v = e.permute(0, 1, 4, 2, 5, 6, 8, 3, 7).reshape(m, D, D).mT
    k, v = k.double(), v.double()                                  # [m, token, channel]
    if lean:
        ck, sk, zk, rv, sv, zv = meta.unbind(1)
        k = (k * sk[:, None] + zk[:, None]) * ck[:, :, None]
        v = (v * sv[:, :, None] + zv[:, :, None]) * rv[:, None]
    else:
        rk, ck, sk, zk, rv, cv, sv, zv = meta.unbind(1)
        k = (k * sk[:, None] + zk[:, None]) * rk[:, None] * ck[:, :, None]
        v = (v * sv[:, :, None] + zv[:, :, None]) * rv[:, None] * cv[:, :, None]
    for step in (1, 2, 4, 8, 16, 32, 64):                          # the rotation as butterflies
        k, v = (torch.stack((x.reshape(m, D, -1, 2, step)[..., 0, :] + x.reshape(m, D, -1, 2, step)[..., 1, :],
                             x.reshape(m, D, -1, 2, step)[..., 0, :] - x.reshape(m, D, -1, 2, step)[..., 1, :]),
                            -2).reshape(m, D, D) for x in (k, v))
    return k / math.sqrt(D), v / math.sqrt(D)


def _sequence64(s, i, h):
    """K and V [token, channel] of sequence i's cached tokens, kv-head h."""
    n = int(s["lens"][i])
    parts = [s["ws"][i, h, :, : n % D].double()]
    if n >= D:
        k, v = _tile64(s["cache"][s["tables"][i, : n // D].long(), h], s["case"]["preset"])
        parts.insert(0, torch.stack((k.reshape(-1, D), v.reshape(-1, D))))
    return torch.cat(parts, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "axes":
        out = []
        rot = 2 * len(s["axes"])
        turn = torch.zeros(case["n"], D // 2, dtype=torch.float64, device="cuda")
        for i, a in enumerate(s["axes"]):
            turn[:, i] = s["pos"][a].double() * s["inv_freq"][i].double()
        w = torch.polar(torch.ones_like(turn), turn)[:, None]
        first = torch.arange(D // 2, device="cuda")
        pair = (2 * first, 2 * first + 1) if case["interleaved"] else (
            torch.where(first < rot // 2, first, rot // 2 + first),
            torch.where(first < rot // 2, first + rot // 2, rot // 2 + first))
        if not case["interleaved"]:  # the channels behind the rotated ones, paired as they come
            rest = torch.arange(rot, D, device="cuda")
            pair = tuple(torch.cat((p[: rot // 2], r)) for p, r in zip(pair, (rest[0::2], rest[1::2])))
        for x, g in ((s["q"], s["q_w"]), (s["k"], s["k_w"])):
            x = x.double()
            if g is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * g.double()
            z = torch.complex(x[..., pair[0]], x[..., pair[1]]) * w
            y = torch.empty_like(x)
            y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
            out.append(y)
        return out + [s["v"].double()]
    if op == "weigh":
        hq, hkv = case["hq"], case["hkv"]
        group = hq // hkv
        out = torch.zeros(case["seqs"], hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((case["seqs"], hq), -math.inf, dtype=torch.float64, device="cuda")
        weights = s["weights"].double()
        for i, n in enumerate(s["lens"].tolist()):
            for h in range(hkv if n else 0):
                k, v = _sequence64(s, i, h)
                x = s["q"][i, h * group:(h + 1) * group].double() @ k.T / math.sqrt(D)
                lse[i, h * group:(h + 1) * group] = torch.logsumexp(x, 1)
                p = torch.softmax(x, 1)
                out[i, h * group:(h + 1) * group] = p @ v
                t = -(-n // D)
                mass = torch.zeros(t * D, dtype=torch.float64, device="cuda")
                mass[:n] = p.sum(0)
                weights[i, h, :t] = case["decay"] * weights[i, h, :t] + mass.reshape(t, D).sum(1)
        return {"out": out, "lse": lse, "weights": weights}
    weights = s["weights"].double().cpu()
    out = torch.zeros_like(weights)
    for i, (n, budget) in enumerate(zip(s["lens"].tolist(), s["budgets"].tolist())):
        t = n // D
        b = min(t, budget)
        first = min(case["first"], b)
        last = min(case["last"], b - first)
        for h in range(case["hkv"]):
            row = weights[i, h].tolist()
            order = sorted(range(first, t - last), key=lambda j: (-row[j], j))[: b - first - last]
            stay = {j for j in order if j < b - last}
            late = sorted(j for j in order if j >= b - last)
            new = [row[j] if j < first or j in stay else row[late.pop(0)] for j in range(b - last)]
            new += row[t - last:t] + row[t:t + 1]
            out[i, h, : len(new)] = torch.tensor(new, dtype=torch.float64)
    return {"kept": None, "lengths": None, "weights": out.cuda(), "cache": None}
