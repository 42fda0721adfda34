"""Cases of the operators around a verify step over the quantized cache: what a
serving loop with drafted tokens runs between the model's projections and its next
step, and the reading back of cached tokens.

  rope    the fused projection's q, k, v rows to per-head normalised, rotated fp16 q and
          k (and fp16 v), the layout that the attention and append calls take
  tree    attention of drafted tokens (a tree, or a chain) over the packed cache, the
          workspace and the drafted tokens themselves
  append  the accepted drafted tokens into the workspace
  read    cached tokens back as plain K and V rows

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
LOG2E = 1.4426950408889634


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence: the latency of a plain decode step's rotation
        dict(name="rope decode 1", op="rope", n=1, hq=64, hkv=8, dtype="fp16", norm=True, rotary=128, interleaved=False,
             fused=True, far=4096),
        # the drafted tokens of a batch in bf16, far positions, half of each head rotated
        dict(name="rope verify 509", op="rope", n=509, hq=40, hkv=8, dtype="bf16", norm=True, rotary=64,
             interleaved=True, fused=True, far=131072),
        # a prefill batch out of the fused projection
        dict(name="rope prefill 65536", op="rope", n=65536, hq=64, hkv=8, dtype="fp16", norm=True, rotary=128,
             interleaved=False, fused=True, far=16384),
        # one short conversation, a small draft: latency
        dict(name="tree 1x1000 t5", op="tree", preset="k4v2", hq=64, hkv=8, seqs=1, lo=1000, hi=1000, t_lo=5, t_hi=5,
             chain=False, softcap=0.0, window=0, slopes=False),
        # the decode batch with eight drafted tokens a sequence
        dict(name="tree 64x16384 t8", op="tree", preset="k4v2", hq=64, hkv=8, seqs=64, lo=16384, hi=16384, t_lo=8,
             t_hi=8, chain=False, softcap=0.0, window=0, slopes=False),
        # few long sequences, 2-bit keys: the context split over the GPU
        dict(name="tree 4x131072 t4 k2v2", op="tree", preset="k2v2", hq=64, hkv=8, seqs=4, lo=131072, hi=131072, t_lo=4,
             t_hi=4, chain=True, softcap=0.0, window=0, slopes=False),
        # a ragged batch, drafts of odd lengths, capped and distance-biased scores in a window
        dict(name="tree ragged capped window", op="tree", preset="k4v4", hq=40, hkv=8, seqs=37, lo=1024, hi=32768,
             t_lo=1, t_hi=13, chain=False, softcap=30.0, window=4096, slopes=True),
        # wide trees over middling contexts: bound by arithmetic
        dict(name="tree 16x4096 t64", op="tree", preset="k4v2l", hq=64, hkv=8, seqs=16, lo=3900, hi=4200, t_lo=64,
             t_hi=64, chain=False, softcap=0.0, window=0, slopes=False),
        # one accepted token of few sequences: latency
        dict(name="append 4 t1", op="append", preset="k4v2", hkv=8, seqs=4, lo=100, hi=5000, t=1, accept=1),
        # the ragged serving batch, some of eight drafted tokens accepted (none at times)
        dict(name="append 256 t8", op="append", preset="k4v2", hkv=8, seqs=256, lo=1024, hi=32768, t=8, accept=6),
        # odd ranges of a few sequences, ending inside a tile and in the workspace
        dict(name="read 3 ragged", op="read", preset="k4v4", hkv=8, seqs=3, lo=200, hi=3000, part=0.7, dtype="bf16"),
        # a whole prefill batch read back, e.g. to hand it to another engine
        dict(name="read 16x16384", op="read", preset="k4v2", hkv=8, seqs=16, lo=16384, hi=16384, part=1.0, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "append", "read"])
    hq, hkv = rng.choice([(64, 8), (40, 8), (32, 8), (28, 4), (8, 1), (6, 2), (8, 8)])
    preset = rng.choice(sorted(PRESETS))
    if op == "rope":
        dtype = rng.choice(sorted(DTYPES))
        return dict(op=op, n=_log(rng, 1, 65536 if dtype != "fp32" else 30000), hq=hq, hkv=hkv, dtype=dtype,
                    norm=rng.random() < 0.7, rotary=rng.choice([32, 64, 128, 128]), interleaved=rng.random() < 0.4,
                    fused=rng.random() < 0.7, far=_log(rng, 64, 1000000))
    if op == "tree":
        hi = _log(rng, 1, 131072)
        lo = max(0, hi - rng.choice([0, 1, hi // 3, hi - 1]))
        t_hi = _log(rng, 1, 64)
        # no more work or context than the largest listed cases
        most = max(1, min(256, (1 << 20) // (hi + 64), (1 << 23) // ((hi + 64) * t_hi)))
        return dict(op=op, preset=preset, hq=hq, hkv=hkv, seqs=_log(rng, 1, most), lo=lo, hi=hi,
                    t_lo=rng.choice([1, t_hi]), t_hi=t_hi, chain=rng.random() < 0.3,
                    softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                    slopes=rng.random() < 0.3)
    if op == "append":
        t = _log(rng, 1, 64)
        return dict(op=op, preset=preset, hkv=hkv, seqs=_log(rng, 1, 256), lo=rng.choice([0, 100]),
                    hi=_log(rng, 200, 131072), t=t, accept=rng.randint(1, t))
    hi = _log(rng, 1, 131072)
    return dict(op=op, preset=preset, hkv=hkv, seqs=_log(rng, 1, max(1, min(256, 262144 // hi))), lo=max(1, hi // 3),
                hi=hi, part=rng.choice([1.0, rng.uniform(0.05, 1.0)]), dtype=rng.choice(["fp16", "bf16", "fp32"]))


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], spread over its logarithm where it is wide; the case alone fixes them."""
    u = [(0.5 + 0.6180339887498949 * i) % 1.0 for i in range(n)]
    if hi > 10 * max(lo, 1):
        return [min(hi, max(lo, int(round(max(lo, 1) * math.exp(x * math.log(hi / max(lo, 1))))))) for x in u]
    return [lo + int(x * (hi - lo + 1)) if hi > lo else lo for x in u]


def _record_bytes(preset):
    kb, vb, lean = PRESETS[preset]
    return D * D * (kb + vb) // 8 + (1536 if lean else 2048)


# ------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


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


def _paged(case, g, lens):
    """Cache, block tables over a random permutation of its blocks (entries behind a sequence's last are -1), workspace."""
    full = [n // D for n in lens]
    width = max(1, max(-(-n // D) for n in lens) + 1)
    blocks = sum(full) + 3
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    fulls = torch.tensor(full, device="cuda")
    tables[torch.arange(width, device="cuda")[None] < fulls[:, None]] = perm[: sum(full)]
    cache = _cache(g, case["preset"], blocks, case["hkv"])
    ws = _normal(g, len(lens), case["hkv"], 2, D, D) * torch.exp(0.4 * _normal(g, len(lens), case["hkv"], 2, 1, D))
    return dict(cache=cache, tables=tables, ws=ws.half(), width=width, blocks=blocks, lens=_i32(lens))


def _trees(case, counts, seed):
    """Ancestor words (bit j: drafted token j of the same sequence is seen) and depths of random trees."""
    import random

    r = random.Random(seed * 7919 + 5)
    words, depths = [], []
    for n in counts:
        w, d = [], []
        for p in range(n):
            up = p - 1 if case["chain"] else r.randint(max(-1, p // 2 - 2), p - 1)
            w.append((w[up] if up >= 0 else 0) | 1 << p)
            d.append(d[up] + 1 if up >= 0 else 0)
        words += w
        depths += d
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda"), depths


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "rope":
        n, hq, hkv, t = case["n"], case["hq"], case["hkv"], DTYPES[case["dtype"]]
        if case["fused"]:
            qkv = _normal(g, n, (hq + 2 * hkv) * D).mul_(1.7).to(t)
            s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
        else:
            s["q"], s["k"], s["v"] = (_normal(g, n, h, D).mul_(1.7).to(t) for h in (hq, hkv, hkv))
        s["q_w"], s["k_w"] = ((1 + 0.2 * _normal(g, D)).to(t) if case["norm"] else None for _ in range(2))
        s["pos"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        half = case["rotary"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        s["out"] = [torch.empty(n, h, D, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
        s["blocks"] = s["width"] = 1
    elif op == "tree":
        lens, counts = _spread(case["seqs"], case["lo"], case["hi"]), _spread(case["seqs"], case["t_lo"], case["t_hi"])
        s |= _paged(case, g, lens)
        cu, n = _cu(counts), sum(counts)
        s["cu"], s["max_t"], s["max_len"] = _i32(cu), max(counts), max(lens)
        s["mask"], depths = _trees(case, counts, seed)
        at = [lens[i] + depths[j] for i in range(len(counts)) for j in range(cu[i], cu[i + 1])]
        s["pos"] = _i32(at)
        s["q"] = _normal(g, n, case["hq"], D).half()
        s["k"], s["v"] = ((_normal(g, n, case["hkv"], D) * torch.exp(0.4 * _normal(g, 1, case["hkv"], D))).half()
                          for _ in range(2))
        s["slopes"] = None
        if case["slopes"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["hq"] + 1, device="cuda") / case["hq"])
        s["out"] = torch.empty_like(s["q"])
    elif op == "append":
        # lengths and accepted counts that complete no tile: what a completed tile's record
        # holds is the tile quantization's output, and steps between codes there decide ties
        t, seqs = case["t"], case["seqs"]
        lens = [n - n % D + n % D % (D - t) for n in _spread(seqs, case["lo"], case["hi"])]
        s |= _paged(case, g, lens)
        s["cu"] = _i32(_cu([t] * seqs))
        s["k"], s["v"] = (_normal(g, seqs * t, case["hkv"], D).half() for _ in range(2))
        s["n_acc"] = torch.randint(0 if t > 1 else 1, case["accept"] + 1, (seqs,), generator=g, device="cuda",
                                   dtype=torch.int32)
        path = torch.rand(seqs, t, generator=g, device="cuda").argsort(1)[:, : case["accept"]]
        s["acc"] = path.sort(1).values.to(torch.int32).contiguous()
        s["lens_out"] = torch.empty_like(s["lens"])
    else:
        lens = _spread(case["seqs"], case["lo"], case["hi"])
        s |= _paged(case, g, lens)
        counts = [max(1, int(n * case["part"])) for n in lens]
        first = [int((n - c) * 0.37) if i % 2 else n - c for i, (n, c) in enumerate(zip(lens, counts))]
        s["first"], s["cu"], s["max_len"] = _i32(first), _i32(_cu(counts)), max(lens)
        s["out"] = [torch.empty(sum(counts), case["hkv"], D, dtype=DTYPES[case["dtype"]], device="cuda")
                    for _ in range(2)]
    if own:
        import kv_cache_quantization_x128_gb300 as kv

        s["meta"] = kv.make_meta(case["hkv"], case.get("hq", case["hkv"]), s["blocks"], s["width"],
                                 preset=case.get("preset", "k4v2"))
        if op == "tree":
            s["scratch"] = torch.empty(kv.tree_scratch_bytes(s["meta"], case["seqs"], s["max_t"]), dtype=torch.uint8,
                                       device="cuda")
    return s


# ------------------------------------------------------------------------ the passes
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "tree": _own_tree, "append": _own_append, "read": _own_read}[op](s)
    return {"rope": _rope, "tree": _tree, "append": _append, "read": _read}[op](s)


def _own_rope(s):
    import kv_cache_quantization_x128_gb300 as kv

    c = s["case"]
    kv.kvarn_qk_norm_rope(s["q"], s["k"], s["v"], s["pos"], *s["out"], s["meta"], q_weight=s["q_w"], k_weight=s["k_w"],
                          norm_eps=1e-6, inv_freq=s["inv_freq"], interleaved=c["interleaved"])
    return s["out"]


def _own_tree(s):
    import kv_cache_quantization_x128_gb300 as kv

    c = s["case"]
    kv.kvarn_tree_attention(s["q"], s["k"], s["v"], None if c["chain"] else s["mask"], s["cu"], s["lens"], s["max_t"],
                            s["tables"], s["cache"], s["ws"], s["out"], s["scratch"], s["meta"], positions=s["pos"],
                            softcap=c["softcap"], window=c["window"], slopes=s["slopes"])
    return s["out"]


def _own_append(s):
    import kv_cache_quantization_x128_gb300 as kv

    kv.kvarn_append_tokens(s["k"], s["v"], s["cu"], s["lens"], s["lens_out"], s["tables"], s["ws"], s["cache"], s["meta"],
                           accepted=s["acc"], n_accepted=s["n_acc"])
    return {"workspace": s["ws"], "lengths": s["lens_out"]}


def _own_read(s):
    import kv_cache_quantization_x128_gb300 as kv

    kv.kvarn_read_tokens(s["cache"], s["ws"], s["tables"], s["lens"], s["cu"], *s["out"], s["meta"], first=s["first"])
    return s["out"]


def _rope(s):
    c = s["case"]
    rot, half = c["rotary"], c["rotary"] // 2
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
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


def _tree(s):
    c = s["case"]
    hq, hkv, t = c["hq"], c["hkv"], s["max_t"]
    lens, cu = s["lens"].long(), s["cu"].long()
    n = lens.numel()
    j = torch.arange(t, device="cuda")
    live = j[None] < (cu[1:] - cu[:-1])[:, None]
    idx = (cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][idx].float().reshape(n, t, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, D)
    kc, vc, at = _cached(s)
    k = torch.cat((kc, s["k"][idx].float().transpose(1, 2)), 2)
    v = torch.cat((vc, s["v"][idx].float().transpose(1, 2)), 2)
    del kc, vc
    pq = s["pos"][idx].long()
    seen = torch.cat(((at[None] < lens[:, None])[:, None].expand(n, t, -1),
                      ((s["mask"][idx][:, :, None] >> j) & 1).bool() & live[:, None]), 2)
    far = pq[:, :, None] - torch.cat((at[None].expand(n, -1), pq), 1)[:, None]
    if c["window"]:
        seen = seen & (far < c["window"])
    x = (q @ k.mT).unflatten(2, (hq // hkv, t)) / math.sqrt(D)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(1, hkv, -1, 1, 1) * far[:, None, None].float()
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    del x
    y = p.flatten(2, 3) @ v / p.flatten(2, 3).sum(-1, keepdim=True).clamp(min=1e-30)
    y = y.unflatten(2, (hq // hkv, t)).permute(0, 3, 1, 2, 4).reshape(n, t, hq, D)
    s["out"].copy_(y[live])
    return s["out"]


def _append(s):
    lens, ws = s["lens"].long(), s["ws"]
    n, hkv, width = ws.shape[0], ws.shape[1], s["acc"].shape[1]
    i = torch.arange(width, device="cuda")
    row, i = torch.nonzero(i[None] < s["n_acc"][:, None], as_tuple=True)
    src = s["cu"].long()[row] + s["acc"].long()[row, i]
    ws[row, :, 0, (lens[row] + i) % D] = s["k"][src]
    ws[row, :, 1, (lens[row] + i) % D] = s["v"][src]
    s["lens_out"].copy_(s["lens"] + s["n_acc"])
    return {"workspace": ws, "lengths": s["lens_out"]}


def _read(s):
    k, v, _ = _cached(s)
    cu = s["cu"].long()
    total = s["out"][0].shape[0]
    at = torch.arange(total, device="cuda")
    row = torch.searchsorted(cu, at, right=True) - 1
    pos = s["first"].long()[row] + at - cu[row]
    for x, out in zip((k, v), s["out"]):
        out.copy_(x[row, :, pos])
    return s["out"]


# ------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "rope":
        n, heads = case["n"], case["hq"] + 2 * case["hkv"]
        size = DTYPES[case["dtype"]].itemsize
        return {"bytes": n * heads * D * (size + 2) + 4 * n, "flops": n * (heads - case["hkv"]) * D * 8}
    rec = _record_bytes(case["preset"])
    row = case["hkv"] * D * 4  # fp16 K and V of one token
    if op == "append":
        n = case["seqs"] * (case["accept"] + (case["t"] == 1)) / (1 if case["t"] == 1 else 2)
        return {"bytes": 2 * n * row + 12 * case["seqs"], "flops": 0}
    lens = _spread(case["seqs"], case["lo"], case["hi"])
    if op == "tree":
        total = flops = 0
        for n, t in zip(lens, _spread(case["seqs"], case["t_lo"], case["t_hi"])):
            deep = t if case["chain"] else 1 + math.log2(t)
            begin = max(0, n - case["window"] + 1) if case["window"] else 0
            tiles = n // D - min(n // D, begin // D)
            total += tiles * case["hkv"] * rec + (n % D + t) * row + t * case["hq"] * D * 4 + 8 * t
            flops += 4 * D * case["hq"] * t * (n - begin + deep)
        return {"bytes": total, "flops": flops}
    total = 0
    for i, n in enumerate(lens):
        c = max(1, int(n * case["part"]))
        total += c * case["hkv"] * (rec / D + 2 * D * DTYPES[case["dtype"]].itemsize)
    return {"bytes": total, "flops": sum(lens) * case["part"] * case["hkv"] * D * 2 * 10}


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
    if op == "rope":
        out = []
        turn = torch.zeros(case["n"], D // 2, dtype=torch.float64, device="cuda")
        rot = case["rotary"]
        turn[:, : rot // 2] = s["pos"].double()[:, None] * s["inv_freq"].double()
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
    if op == "append":
        ws, lens = s["ws"].double(), s["lens"].tolist()
        for i, (n, a) in enumerate(zip(lens, s["n_acc"].tolist())):
            for x in range(a):
                src = int(s["cu"][i]) + int(s["acc"][i, x])
                ws[i, :, 0, (n + x) % D], ws[i, :, 1, (n + x) % D] = s["k"][src].double(), s["v"][src].double()
        return {"workspace": ws, "lengths": None}
    if op == "read":
        total, hkv = s["out"][0].shape[0], case["hkv"]
        out = torch.empty(2, total, hkv, D, dtype=torch.float64, device="cuda")
        cu, first = s["cu"].tolist(), s["first"].tolist()
        for i in range(case["seqs"]):
            for h in range(hkv):
                out[:, cu[i]:cu[i + 1], h] = _sequence64(s, i, h)[:, first[i]: first[i] + cu[i + 1] - cu[i]]
        return [out[0], out[1]]
    hq, hkv = case["hq"], case["hkv"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    out = torch.zeros(cu[-1], hq, D, dtype=torch.float64, device="cuda")
    group = hq // hkv
    for i in range(case["seqs"]):
        a, b, n = cu[i], cu[i + 1], lens[i]
        pq = s["pos"][a:b].double()
        word = s["mask"][a:b]
        bits = torch.stack([(word >> j) & 1 for j in range(b - a)], 1).bool()
        seen = torch.cat((torch.ones(b - a, n, dtype=torch.bool, device="cuda"), bits), 1)
        gap = pq[:, None] - torch.cat((torch.arange(n, dtype=torch.float64, device="cuda"), pq))[None]
        if case["window"]:
            seen = seen & (gap < case["window"])
        for h in range(hkv):
            kv = torch.cat((_sequence64(s, i, h), torch.stack((s["k"][a:b, h], s["v"][a:b, h])).double()), 1)
            for m in range(h * group, h * group + group):
                x = s["q"][a:b, m].double() @ kv[0].T / math.sqrt(D)
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][m].double() * gap
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                out[a:b, m] = torch.softmax(x, 1) @ kv[1]
    return out
