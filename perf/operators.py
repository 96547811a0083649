"""Cases of the rotary-position, 8-bit cache append and 8-bit cache attention operators, their plain forms in torch,
and their definitions in 64 bits."""
import math

import torch

own = False

# Rotary pairs per axis (time, height, width) of the framework's head sizes.
PAIRS = {128: (22, 21, 21), 64: (12, 10, 10)}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
THETA = 10000.0


def listed():
    return [
        # q of one latent block (3 frames of the 30x52 grid, 40 heads), before attention
        {"name": "rope_block", "op": "rope", "tokens": 4680, "heads": 40, "dim": 128, "dtype": "bf16", "half": False,
         "inverse": False, "far": False},
        # one new token of one stream, far into a long stream: latency
        {"name": "rope_token", "op": "rope", "tokens": 1, "heads": 40, "dim": 128, "dtype": "bf16", "half": False,
         "inverse": False, "far": True},
        # the gradient of q and k in training on one 45x80 frame and an odd remainder, fp32, split-half pairs
        {"name": "rope_grad", "op": "rope", "tokens": 3601, "heads": 24, "dim": 64, "dtype": "fp32", "half": True,
         "inverse": True, "far": False},
        # one latent block of one stream enters its cache behind a ragged tail
        {"name": "append_block", "op": "append", "seqs": 1, "new": 4680, "old": 9403, "heads": 40, "dim": 128,
         "page": 64, "dtype": "bf16", "half": False, "ragged": False},
        # one token for each of 16 streams: partly filled pages whose scales may grow
        {"name": "append_token", "op": "append", "seqs": 16, "new": 1, "old": 1563, "heads": 8, "dim": 128, "page": 64,
         "dtype": "bf16", "half": True, "ragged": True},
        # ragged pieces of 5 streams at once, small heads and pages
        {"name": "append_ragged", "op": "append", "seqs": 5, "new": 777, "old": 300, "heads": 12, "dim": 64, "page": 32,
         "dtype": "fp16", "half": False, "ragged": True},
        # one latent block's queries over [sink | 2 window blocks | block], every key visible: the stream's own shape
        {"name": "attn_block", "op": "attn", "seqs": 1, "q": 4680, "kv": 15600, "heads": 40, "group": 1, "dim": 128,
         "page": 64, "dtype": "bf16", "causal": 0, "ragged": False},
        # one query token for each of 16 streams over long caches
        {"name": "attn_token", "op": "attn", "seqs": 16, "q": 1, "kv": 14040, "heads": 40, "group": 1, "dim": 128,
         "page": 64, "dtype": "bf16", "causal": 1, "ragged": True},
        # one query token of one stream over a short cache, grouped heads: latency
        {"name": "attn_token_one", "op": "attn", "seqs": 1, "q": 1, "kv": 1561, "heads": 40, "group": 5, "dim": 128,
         "page": 64, "dtype": "bf16", "causal": 1, "ragged": False},
        # one query token of one stream over a very long cache of few key heads: the work is split along the keys
        {"name": "attn_token_long", "op": "attn", "seqs": 1, "q": 1, "kv": 187203, "heads": 16, "group": 8, "dim": 128,
         "page": 128, "dtype": "fp16", "causal": 1, "ragged": False},
        # prompts of 4 streams in one call, token-causal, grouped heads of 64
        {"name": "attn_causal", "op": "attn", "seqs": 4, "q": 1013, "kv": 4090, "heads": 16, "group": 4, "dim": 64,
         "page": 32, "dtype": "fp16", "causal": 1, "ragged": True},
        # whole frames under the block-causal mask (frames of the 30x52 grid), a context of 5 frames
        {"name": "attn_frames", "op": "attn", "seqs": 2, "q": 4680, "kv": 7800, "heads": 16, "group": 2, "dim": 128,
         "page": 128, "dtype": "bf16", "causal": 1560, "ragged": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    dim = rng.choice([64, 128])
    page = rng.choice([32, 64, 128])
    if op == "rope":
        heads = rng.choice([1, 8, 24, 40])
        return {"op": op, "tokens": _log(rng, 1, 4800 * 40 // heads), "heads": heads, "dim": dim,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "half": rng.random() < 0.5,
                "inverse": rng.random() < 0.5, "far": rng.random() < 0.3}
    if op == "append":
        seqs, heads = _log(rng, 1, 32), rng.choice([1, 4, 8, 40])
        return {"op": op, "seqs": seqs, "new": _log(rng, 1, max(1, 4680 * 40 // (heads * seqs))),
                "old": _log(rng, 1, 4000), "heads": heads, "dim": dim, "page": page,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "half": rng.random() < 0.5,
                "ragged": rng.random() < 0.6}
    group = rng.choice([1, 2, 4, 5, 8])
    heads = group * rng.choice([1, 2, 4, 8])
    causal = rng.choice([0, 1, 1, 1560, 240])
    if rng.random() < 0.5:      # single tokens and short drafts
        seqs, q = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 3, 5, 8])
        kv = _log(rng, 16, 200000)
        while seqs * kv * heads > 16 * 14040 * 40:
            kv = (kv + 1) // 2
    else:                       # prompts and blocks
        seqs, q = _log(rng, 1, 4), _log(rng, 9, 4800)
        kv = max(q, _log(rng, 64, 15600))
        while seqs * q * kv * heads > 4680 * 15600 * 40:
            q = (q + 1) // 2
    return {"op": op, "seqs": seqs, "q": q, "kv": max(kv, q), "heads": heads, "group": group, "dim": dim, "page": page,
            "dtype": rng.choice(["bf16", "fp16"]), "causal": causal, "ragged": rng.random() < 0.6}


def _lens(case, top, salt):
    """Lengths of the case's sequences: all `top`, or ragged ones from 1 to `top` with the first at `top`."""
    n = case["seqs"]
    if not case["ragged"]:
        return [top] * n
    return [max(1, top - (i * (salt + top // 7)) % max(1, top)) for i in range(n)]


def _plan(case):
    """(new or query lengths, key lengths before or at the call, pages of a sequence)."""
    if case["op"] == "append":
        new, old = _lens(case, case["new"], 3), _lens(case, case["old"], 5)
        return new, old, -(-max(n + o for n, o in zip(new, old)) // case["page"])
    q, kv = _lens(case, case["q"], 3), _lens(case, case["kv"], 5)
    kv = [max(a, b) for a, b in zip(q, kv)]
    return q, kv, -(-max(kv) // case["page"])


def _positions(n, far, gen, dev):
    """(time, height, width) of n tokens in row-major order of a 30x52 grid, as a stream numbers them."""
    i = torch.arange(n, device=dev)
    start = int(torch.randint(3, 90000 if far else 600, (1,), generator=gen, device=dev))
    return torch.stack([start + i // 1560, i % 1560 // 52, i % 52], 1).to(torch.int32)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    dt = DTYPES[case["dtype"]]
    d = case["dim"]
    if case["op"] == "rope":
        n = case["tokens"]
        return {"case": case, "x": rnd(n, case["heads"], d).to(dt), "pos": _positions(n, case["far"], gen, dev)}
    rows, keys, width = _plan(case)
    b, page = case["seqs"], case["page"]
    heads = case["heads"] // case.get("group", 1)
    cu = torch.tensor([0] + rows, device=dev).cumsum(0).to(torch.int32)
    pages = b * width
    table = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).view(b, width)
    shape = (pages, heads, page, d)
    # e4m3 codes as an append leaves them: the largest of a page in (224, 448], scales of one page's spread
    spread = 100.0
    codes = [(rnd(*shape) * spread).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-8, -5, shape[:2], generator=gen, device=dev).float()) for _ in range(2)]
    lens = torch.tensor(keys, device=dev, dtype=torch.int32)
    state = {"case": case, "k_pages": codes[0], "v_pages": codes[1], "k_scale": scales[0], "v_scale": scales[1],
             "table": table, "lens": lens, "cu": cu, "max_rows": max(rows), "max_keys": max(keys)}
    n = sum(rows)
    if case["op"] == "append":
        # values grow over time in some heads, so that partly filled pages have to raise their scale
        grow = torch.exp2(torch.randint(-1, 3, (1, heads, 1), generator=gen, device=dev).float())
        state |= {"k": (rnd(n, heads, d) * grow).to(dt), "v": (rnd(n, heads, d) * grow).to(dt),
                  "pos": _positions(n, False, gen, dev)}
    else:
        state["q"] = rnd(n, case["heads"], d).to(dt)
    return state


def _angles(pos, pairs, dtype):
    """[T, pairs] angles in 64 bits: axis a's j-th pair turns by pos * theta^(-j / pairs_a)."""
    axis = torch.cat([torch.full((p,), i, dtype=torch.long) for i, p in enumerate(pairs)]).to(pos.device)
    freq = torch.cat([THETA ** (-torch.arange(p, dtype=torch.float64) / p) for p in pairs]).to(pos.device)
    ang = pos.to(torch.float64)[:, axis] * freq
    return torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def _rotate(x, pos, pairs, half, inverse):
    """x [T, H, d] in fp32, rotated."""
    c, s = _angles(pos, pairs, torch.float32)
    c, s = c[:, None], (-s if inverse else s)[:, None]
    n = sum(pairs)
    a, b = (x[..., :n], x[..., n:2 * n]) if half else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
    u, w = a * c - b * s, a * s + b * c
    y = torch.cat([u, w], -1) if half else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _append_plain(s, x, pages, scale):
    """Writes x [N, H, d] (fp32) into the e4m3 pages, one power-of-two scale a (page, head)."""
    case, page = s["case"], s["case"]["page"]
    tok = torch.arange(x.shape[0], device=x.device)
    seq = torch.searchsorted(s["cu"].long(), tok, right=True) - 1
    at = s["lens"].long()[seq] + tok - s["cu"].long()[seq]
    pg, off = s["table"].long()[seq, at // page], at % page
    amax = torch.zeros_like(scale).index_reduce_(0, pg, x.abs().amax(-1), "amax")
    new = torch.zeros(pages.shape[0], page, dtype=torch.bool, device=x.device).index_put((pg, off), torch.ones((), dtype=torch.bool, device=x.device))
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-64)
    need = torch.exp2(k.float())
    touched = new.any(1)
    fresh = torch.where(new[:, :1], need, torch.maximum(scale, need))
    fresh = torch.where(touched[:, None], fresh, scale)
    first = torch.where(touched, new.float().argmax(1), 0)
    old = torch.arange(page, device=x.device) < first[:, None]
    vals = pages.view(torch.float8_e4m3fn).float()
    moved = (vals * (scale / fresh)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(old[:, None, :, None], moved, pages)
    codes[pg, :, off] = (x / fresh[pg][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    pages.copy_(codes)
    scale.copy_(fresh)


def _attn_plain(s):
    case = s["case"]
    b, h, g, d, page = case["seqs"], case["heads"], case["group"], case["dim"], case["page"]
    hk, nq, dt = h // g, s["max_rows"], DTYPES[case["dtype"]]
    table, cu, kv = s["table"].long(), s["cu"].long(), s["lens"].long()
    dense = lambda p, c: (p.view(torch.float8_e4m3fn)[table].float() * c[table][..., None, None]).transpose(1, 2).reshape(b, hk, -1, d)  # noqa: E731
    k, v = dense(s["k_pages"], s["k_scale"]), dense(s["v_pages"], s["v_scale"])
    r = torch.arange(nq, device=k.device)
    n = (cu[1:] - cu[:-1])
    rows = (cu[:-1, None] + r).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float() * (1.0 / math.sqrt(d))                     # [B, nq, H, d]
    q = q.view(b, nq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * nq, d)
    sc = q @ k.transpose(-1, -2)
    j = torch.arange(k.shape[2], device=k.device)
    lim = kv[:, None].expand(b, nq)
    if case["causal"]:
        lim = torch.minimum(lim, (kv - n)[:, None] + (r // case["causal"] + 1) * case["causal"])
    seen = (j < lim[..., None])[:, None, None]                          # [B, 1, 1, nq, L]
    sc = sc.view(b, hk, g, nq, -1).masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    z = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, g * nq, -1) @ v).view(b, hk, g, nq, d) / torch.where(z == 0, torch.ones_like(z), z)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, nq, h, d).to(dt)
    return o[r < n[:, None]]


def run(s):
    case = s["case"]
    pairs = PAIRS[case["dim"]]
    if own:
        from streaming_causal_video_timestep_b200 import op_attention_cache_fp8, op_cache_append_fp8, op_rope_axes
        if case["op"] == "rope":
            return op_rope_axes(s["x"], s["pos"], pairs, theta=THETA, half=case["half"], inverse=case["inverse"])
        if case["op"] == "append":
            op_cache_append_fp8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"],
                                s["lens"], s["cu"], s["max_rows"], pos=s["pos"], pairs=pairs, theta=THETA,
                                half=case["half"])
        else:
            return op_attention_cache_fp8(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"],
                                          s["lens"], s["cu"], s["max_rows"], s["max_keys"],
                                          causal_block=case["causal"])
    elif case["op"] == "rope":
        return _rotate(s["x"].float(), s["pos"], pairs, case["half"], case["inverse"]).to(s["x"].dtype)
    elif case["op"] == "append":
        _append_plain(s, _rotate(s["k"].float(), s["pos"], pairs, case["half"], False), s["k_pages"], s["k_scale"])
        _append_plain(s, s["v"].float(), s["v_pages"], s["v_scale"])
    else:
        return _attn_plain(s)
    return {"k": s["k_pages"].view(torch.float8_e4m3fn), "v": s["v_pages"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    d = case["dim"]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * d
        return {"bytes": 2 * n * size + 12 * case["tokens"], "flops": 3 * n}
    rows, keys, _ = _plan(case)
    if case["op"] == "append":
        n = sum(rows) * case["heads"] * d
        pages = sum(-(-(a + o) // case["page"]) - o // case["page"] for a, o in zip(rows, keys))
        return {"bytes": 2 * n * (size + 1) + 12 * sum(rows) + 8 * pages * case["heads"], "flops": 5 * n}
    seen, read = 0, 0
    for n, kv in zip(rows, keys):
        lim = [kv] * n if not case["causal"] else [min(kv, kv - n + (r // case["causal"] + 1) * case["causal"]) for r in range(n)]
        seen += sum(lim)
        read += max(lim)
    hk = case["heads"] // case["group"]
    return {"bytes": 2 * read * hk * (d + 4 / case["page"]) + 2 * sum(rows) * case["heads"] * d * size,
            "flops": 4 * seen * case["heads"] * d}


def exact(case, seed):
    s = prepare(case, seed)
    pairs = PAIRS[case["dim"]]

    def turn(x, sign):
        x = x.double()
        y = x.clone()
        n, j = sum(pairs), 0
        for axis, p in enumerate(pairs):
            for i in range(p):
                a = s["pos"][:, axis].double() * (sign * THETA ** (-i / p))
                lo, hi = (j, n + j) if case["half"] else (2 * j, 2 * j + 1)
                c, w = torch.cos(a)[:, None], torch.sin(a)[:, None]
                y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * w, x[..., lo] * w + x[..., hi] * c
                j += 1
        return y

    if case["op"] == "rope":
        return turn(s["x"], -1.0 if case["inverse"] else 1.0)
    table, cu, lens, page = s["table"].tolist(), s["cu"].tolist(), s["lens"].tolist(), case["page"]
    if case["op"] == "append":
        out = {}
        for name, x in (("k", turn(s["k"], 1.0)), ("v", s["v"].double())):
            code = s[name + "_pages"].view(torch.float8_e4m3fn).double()
            scale = s[name + "_scale"].double()
            for b in range(case["seqs"]):
                t, at, end = cu[b], lens[b], lens[b] + cu[b + 1] - cu[b]
                while at < end:
                    pg, off = table[b][at // page], at % page
                    n = min(page - off, end - at)
                    part = x[t:t + n].transpose(0, 1)                  # [H, n, d]
                    amax = part.abs().amax((1, 2))
                    need = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(min=-64))
                    need = torch.where(amax * 2 <= need * 448, need / 2, need).clamp(min=2.0 ** -64)   # log2 may be an ulp high
                    to = torch.maximum(need, scale[pg]) if off else need
                    if off:
                        code[pg, :, :off] = (code[pg, :, :off] * (scale[pg] / to)[:, None, None]).float().to(torch.float8_e4m3fn).double()
                    code[pg, :, off:off + n] = (part / to[:, None, None]).float().to(torch.float8_e4m3fn).double()
                    scale[pg] = to
                    t, at = t + n, at + n
            out[name], out[name + "_scale"] = code.to(torch.float32).to(torch.float8_e4m3fn), scale
        return out
    g, d = case["group"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(case["seqs"]):
        kv, n = lens[b], cu[b + 1] - cu[b]
        ids = s["table"][b, :-(-kv // page)].long()
        for h in range(case["heads"] // g):
            k, v = ((s[c + "_pages"][ids, h].view(torch.float8_e4m3fn).double() * s[c + "_scale"][ids, h].double()[:, None, None]).reshape(-1, d)[:kv] for c in "kv")
            for r in range(0, n, 1200):
                q = s["q"][cu[b] + r:cu[b] + min(n, r + 1200), h * g:(h + 1) * g].double()
                x = torch.einsum("rgd,kd->rgk", q, k) / math.sqrt(d)
                if case["causal"]:
                    i = torch.arange(r, r + q.shape[0], device=x.device)
                    top = kv - n + (torch.div(i, case["causal"], rounding_mode="floor") + 1) * case["causal"]
                    x = x.masked_fill((torch.arange(kv, device=x.device) >= top[:, None])[:, None], -math.inf)
                out[cu[b] + r:cu[b] + r + q.shape[0], h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
    return out
