"""The operators that serve sigmoid attention from a paged cache, as cases to measure.

Four operators: taking pages for new tokens (``sigattn_paged_reserve``), giving
pages back (``sigattn_paged_release``), rotating and storing new keys and values
(``sigattn_paged_write``), and attention of the new tokens over the cache
(``sigattn_fwd_paged``). ``run`` computes each either in its plain form (torch
operations in 32 bits, rounded once) or, where ``own`` is true, through the
library's entry point. Sizes are this library's own head counts and head sizes
(16 x 128, 12 x 64, 8 x 64) and generic shared-head ones.

Conventions. The cache is [num_pages][Hkv][page_size][d] bf16 for K and for V.
Sequence b holds kv_lens[b] tokens there, the last q_lens[b] of which are the
new ones; its pages are block_table[b][0..]. New token i of a sequence sits at
position p = kv_len - q_len + i and sees N keys: the first p + 1 (causal) or all
kv_len; its weights are sigma(q.k / sqrt(d) - ln N).
"""
import math
import random

import numpy as np
import torch

own = False

PAGES = (16, 32, 64, 128)
HEADS_KV = (1, 2, 4, 8, 12, 16)
GROUPS = (1, 1, 2, 3, 4, 5, 7, 8, 16)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One user, one new token, a short text: the call's own latency.
        dict(name="attend_1_token", op="attend", B=1, Hq=32, Hkv=8, d=128, page=16, causal=True,
             chunks=0, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=1000, lens=1),
        # A full serving batch in its steady state: one token each, ragged texts.
        dict(name="attend_decode_batch", op="attend", B=64, Hq=32, Hkv=8, d=128, page=16, causal=True,
             chunks=0, q_lo=1, q_hi=1, kv_lo=256, kv_hi=8192, lens=2),
        # Few users with very long texts: keys must be split over the SMs.
        dict(name="attend_decode_long", op="attend", B=4, Hq=32, Hkv=4, d=128, page=64, causal=True,
             chunks=0, q_lo=1, q_hi=1, kv_lo=100000, kv_hi=262144, lens=3),
        # A few drafted tokens each, checked at once; no shared heads, d = 64.
        dict(name="attend_draft_tokens", op="attend", B=32, Hq=12, Hkv=12, d=64, page=32, causal=True,
             chunks=32, q_lo=2, q_hi=8, kv_lo=64, kv_hi=4096, lens=4),
        # Two prompts' chunks running beside fourteen users' single tokens.
        dict(name="attend_mixed_chunks", op="attend", B=16, Hq=16, Hkv=4, d=128, page=16, causal=True,
             chunks=2, q_lo=1000, q_hi=1024, kv_lo=1024, kv_hi=8192, lens=5),
        # Long prompts in large chunks: the most arithmetic.
        dict(name="attend_long_prompts", op="attend", B=2, Hq=16, Hkv=16, d=128, page=128, causal=True,
             chunks=2, q_lo=4000, q_hi=4096, kv_lo=8192, kv_hi=16384, lens=6),
        # One step of a serving batch: a token each, a page only now and then.
        dict(name="reserve_decode_batch", op="reserve", B=64, page=16, max_pages=512, chunks=0, q_lo=1, q_hi=1,
             kv_lo=16, kv_hi=8000, lens=7),
        # Many prompts admitted at once.
        dict(name="reserve_prompts", op="reserve", B=256, page=16, max_pages=1024, chunks=256, q_lo=64, q_hi=8192,
             kv_lo=64, kv_hi=8192, lens=8),
        # Rejected draft tokens go back: a few pages over a batch.
        dict(name="release_tails", op="release", B=64, page=16, max_pages=512, kv_lo=32, kv_hi=8000, most=16, lens=9),
        # A batch of finished requests gives all its pages back.
        dict(name="release_finished", op="release", B=512, page=16, max_pages=2048, kv_lo=64, kv_hi=32768, most=32768,
             lens=10),
        # A serving step's tokens, one axis of positions.
        dict(name="write_decode_batch", op="write", T=64, Hq=32, Hkv=8, d=128, page=16, axes=1, pairs=64, adjacent=False,
             far=131072, lens=11),
        # A prompt with images: three axes (time, height, width), rows cut out of one fused projection.
        dict(name="write_image_prompt", op="write", T=16384, Hq=32, Hkv=8, d=128, page=64, axes=3, pairs=64,
             adjacent=False, far=131072, lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "attend", "reserve", "release", "write"))
    lens = rng.randrange(1 << 30)
    if kind == "reserve":
        B, page = _log_int(rng, 1, 1024), rng.choice(PAGES)
        hi = _log_int(rng, 32, 16384 if B <= 256 else 2048)
        return dict(op="reserve", B=B, page=page, max_pages=2 * hi // page + 2, chunks=rng.choice((0, B // 2, B)),
                    q_lo=1, q_hi=hi, kv_lo=1, kv_hi=hi, lens=lens)
    if kind == "release":
        B, page = _log_int(rng, 1, 1024), rng.choice(PAGES)
        hi = _log_int(rng, 32, 16384)
        return dict(op="release", B=B, page=page, max_pages=hi // page + 2, kv_lo=1, kv_hi=hi,
                    most=_log_int(rng, 1, hi), lens=lens)
    if kind == "write":
        Hkv, d = rng.choice(HEADS_KV), rng.choice((64, 128))
        Hq = min(32, Hkv * rng.choice(GROUPS)) // Hkv * Hkv
        return dict(op="write", T=_log_int(rng, 1, 16384 * 48 // max(48, Hq + 2 * Hkv)), Hq=Hq, Hkv=Hkv, d=d,
                    page=rng.choice(PAGES), axes=rng.choice((1, 1, 2, 3)),
                    pairs=rng.choice((d // 2, d // 2, d // 4, 0)),
                    adjacent=rng.random() < 0.5, far=_log_int(rng, 64, 1 << 20), lens=lens)
    while True:
        Hkv, G, d = rng.choice(HEADS_KV), rng.choice(GROUPS), rng.choice((64, 128))
        c = dict(op="attend", B=_log_int(rng, 1, 128), Hq=Hkv * G, Hkv=Hkv, d=d, page=rng.choice(PAGES),
                 causal=rng.random() < 0.7, kv_lo=1, lens=lens)
        form = rng.choice(("tokens", "drafts", "chunks"))
        if form == "tokens":
            c.update(chunks=0, q_lo=1, q_hi=1, kv_hi=_log_int(rng, 16, 262144))
        elif form == "drafts":
            c.update(chunks=c["B"], q_lo=1, q_hi=_log_int(rng, 2, 64), kv_hi=_log_int(rng, 64, 65536))
        else:
            c.update(chunks=rng.randint(1, c["B"]), q_lo=1, q_hi=_log_int(rng, 16, 4096), kv_hi=_log_int(rng, 128, 32768))
        c["kv_lo"] = max(1, c["kv_hi"] // rng.choice((1, 4, 32)))
        q, kv = _lengths(c)
        if (c["Hq"] <= 64 and c["B"] * max(kv) * Hkv * d <= 1 << 28 and c["B"] * c["Hq"] * max(q) * max(kv) <= 1 << 30):
            return c


def _lengths(c):
    """New tokens and cached tokens (new ones included) of every sequence."""
    r = random.Random(c["lens"])
    kv = [_log_int(r, c["kv_lo"], c["kv_hi"]) for _ in range(c["B"])]
    q = [_log_int(r, c["q_lo"], c["q_hi"]) if b < c["chunks"] else 1 for b in range(c["B"])]
    r.shuffle(q)
    return q, [max(a, b) for a, b in zip(q, kv)]


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 4 + 1)
    s = {"case": c}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    def shuffled(n):
        return torch.randperm(n, generator=g, device="cuda").to(torch.int32)

    if c["op"] == "attend":
        q, kv = _lengths(c)
        pages = [_ceil(n, c["page"]) for n in kv]
        num = sum(pages) + sum(pages) // 8 + 1
        order = shuffled(num)
        table = torch.full((c["B"], max(pages)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        s.update(q=normal(sum(q), c["Hq"], c["d"]), k_cache=normal(num, c["Hkv"], c["page"], c["d"]),
                 v_cache=normal(num, c["Hkv"], c["page"], c["d"]), table=table, kv=i32(kv),
                 cu=i32(np.concatenate([[0], np.cumsum(q)]).tolist()), max_q=max(q))
        s["o"] = torch.empty_like(s["q"])
    elif c["op"] == "reserve":
        q, kv = _lengths(c)
        cached = [a - b for a, b in zip(kv, q)]
        have = [_ceil(n, c["page"]) for n in cached]
        need = sum(_ceil(a, c["page"]) - h for a, h in zip(kv, have))
        num = sum(have) + need + 64
        order = shuffled(num)
        table = torch.full((c["B"], c["max_pages"]), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(have):
            table[b, :n] = order[at:at + n]
            at += n
        stack = torch.zeros(num, dtype=torch.int32, device="cuda")
        stack[:num - at] = order[at:]
        T = sum(q)
        e = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s.update(cached=i32(cached), new=i32(q), table=table, stack=stack, count=i32([num - at]), count_out=e(1),
                 cu=e(c["B"] + 1), kv=e(c["B"]), slots=e(T), positions=e(T))
    elif c["op"] == "release":
        kv, keep = _release_lengths(c)
        held = [_ceil(n, c["page"]) for n in kv]
        num = sum(held) + 64
        order = shuffled(num)
        table = torch.full((c["B"], c["max_pages"]), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        stack = torch.zeros(num, dtype=torch.int32, device="cuda")
        stack[:num - at] = order[at:]
        s.update(kv=i32(kv), keep=i32(keep), table=table, stack=stack, count=i32([num - at]),
                 count_out=torch.zeros(1, dtype=torch.int32, device="cuda"))
    else:
        T, d, Hq, Hkv = c["T"], c["d"], c["Hq"], c["Hkv"]
        num = _ceil(T, c["page"]) + 4
        # q, k and v side by side, as one projection writes them
        qkv = normal(T, Hq + 2 * Hkv, d)
        slots = torch.randperm(num, generator=g, device="cuda")[:, None] * c["page"] + torch.arange(c["page"], device="cuda")
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], slots=slots.reshape(-1)[:T].to(torch.int32),
                 k_cache=normal(num, Hkv, c["page"], d), v_cache=normal(num, Hkv, c["page"], d), positions=None,
                 inv_freq=None, pair_axis=None)
        s["q_out"] = torch.empty(T, Hq, d, dtype=torch.bfloat16, device="cuda")
        if c["pairs"]:
            s["positions"] = torch.randint(0, c["far"], (c["axes"], T), generator=g, device="cuda", dtype=torch.int32)
            s["inv_freq"] = 10000.0 ** (-torch.arange(c["pairs"], device="cuda", dtype=torch.float32) / c["pairs"])
            # the first quarter of the pairs turns with axis 0, the rest is shared out evenly
            a = torch.arange(c["pairs"], device="cuda")
            s["pair_axis"] = (torch.clamp((a * 4 // max(1, c["pairs"]) + 1) // 2, max=c["axes"] - 1)).to(torch.int32)
    # zeroed once, as the library asks; enough for any of these calls
    s["workspace"] = torch.zeros(64 << 20 if c["op"] == "attend" else 256, dtype=torch.uint8, device="cuda")
    return s


def _release_lengths(c):
    r = random.Random(c["lens"])
    kv = [_log_int(r, c["kv_lo"], c["kv_hi"]) for _ in range(c["B"])]
    return kv, [max(0, n - r.randint(0, c["most"])) for n in kv]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import sigmoid_attention_b200 as sa
        if c["op"] == "attend":
            sa.sigattn_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["o"], s["cu"], s["kv"], s["table"], s["max_q"],
                                 c["causal"], s["workspace"])
            return s["o"]
        if c["op"] == "reserve":
            sa.sigattn_paged_reserve(s["cached"], s["new"], s["table"], s["stack"], s["count"], s["count_out"], s["cu"],
                                     s["kv"], s["slots"], s["positions"], c["page"], s["workspace"])
            return {k: s[k] for k in ("table", "count_out", "cu", "kv", "slots", "positions")}
        if c["op"] == "release":
            sa.sigattn_paged_release(s["kv"], s["keep"], s["table"], s["stack"], s["count"], s["count_out"], c["page"],
                                     s["workspace"])
            return {k: s[k] for k in ("stack", "count_out")}
        sa.sigattn_paged_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["workspace"], q=s["q"],
                               q_out=s["q_out"], positions=s["positions"], inv_freq=s["inv_freq"],
                               pair_axis=s["pair_axis"], adjacent=c["adjacent"])
        return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}
    return {"attend": _plain_attend, "reserve": _plain_reserve, "release": _plain_release, "write": _plain_write}[c["op"]](s)


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, d, mq = c["B"], c["Hq"], c["Hkv"], c["d"], s["max_q"]
    G = Hq // Hkv
    cu, kv = s["cu"].long(), s["kv"].long()
    table = s["table"].long().clamp(min=0)
    # [B, pages, Hkv, page, d] -> [B, Hkv, keys, d]
    k = s["k_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    v = s["v_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    L = k.shape[2]
    i = torch.arange(mq, device="cuda")
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, mq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * mq, d)
    seen = kv[:, None].expand(B, mq)
    if c["causal"]:
        seen = (kv - (cu[1:] - cu[:-1]))[:, None] + i + 1
    seen = seen.clamp(min=0)[:, None, None, :, None]
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, mq, L).mul_(1 / math.sqrt(d))
    x -= torch.log(seen.clamp(min=1).float())
    w = x.neg_().exp_().add_(1).reciprocal_()
    keys = torch.arange(L, device="cuda")
    w.masked_fill_(keys >= torch.minimum(seen, kv[:, None, None, None, None]), 0)
    o = torch.matmul(w.view(B, Hkv, G * mq, L), v).view(B, Hkv, G, mq, d).permute(0, 3, 1, 2, 4).reshape(B, mq, Hq, d)
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    return o[seq, t - cu[seq]].to(torch.bfloat16)


def _plain_reserve(s):
    c = s["case"]
    ps = c["page"]
    cached, new, F = s["cached"].long(), s["new"].long(), s["count"].long()
    have = (cached + ps - 1) // ps
    need = (cached + new + ps - 1) // ps - have
    off = torch.cumsum(need, 0) - need
    k = torch.arange(c["max_pages"], device="cuda")
    fresh = (k >= have[:, None]) & (k < (have + need)[:, None])
    at = (F - 1 - (off - have)[:, None] - k).clamp(min=0, max=s["stack"].numel() - 1)
    table = torch.where(fresh, s["stack"][at], s["table"])
    cu = torch.cat([torch.zeros_like(F), torch.cumsum(new, 0)])
    t = torch.arange(s["slots"].numel(), device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    pos = cached[seq] + t - cu[seq]
    slots = table[seq, pos // ps] * ps + pos % ps
    i32 = torch.int32
    return {"table": table, "count_out": (F - need.sum()).to(i32), "cu": cu.to(i32), "kv": (cached + new).to(i32),
            "slots": slots.to(i32), "positions": pos.to(i32)}


def _plain_release(s):
    c = s["case"]
    ps = c["page"]
    first, end = (s["keep"].long() + ps - 1) // ps, (s["kv"].long() + ps - 1) // ps
    n = end - first
    off = torch.cumsum(n, 0)
    p = torch.arange(s["stack"].numel(), device="cuda") - s["count"].long()
    seq = torch.searchsorted(off, p.clamp(min=0), right=True).clamp(max=c["B"] - 1)
    k = (first[seq] + p - (off - n)[seq]).clamp(min=0, max=c["max_pages"] - 1)
    stack = torch.where((p >= 0) & (p < off[-1]), s["table"][seq, k], s["stack"])
    return {"stack": stack, "count_out": (s["count"].long() + off[-1:]).to(torch.int32)}


def _turned(x, cos, sin, pairs, adjacent):
    """Rows [T, H, d] with their first 2 * pairs values turned, in the width of cos and sin."""
    x = x.to(cos.dtype)
    if adjacent:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., 2 * pairs:]], -1)


def _plain_write(s):
    c = s["case"]
    slots = s["slots"].long()
    page, off = slots // c["page"], slots % c["page"]
    q, k = s["q"], s["k"]
    if c["pairs"]:
        # far positions: the angles need 64 bits, their cosines and sines do not
        angle = s["positions"][s["pair_axis"].long()].double().t() * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        q = _turned(q, cos, sin, c["pairs"], c["adjacent"]).to(torch.bfloat16)
        k = _turned(k, cos, sin, c["pairs"], c["adjacent"]).to(torch.bfloat16)
    s["k_cache"][page, :, off] = k
    s["v_cache"][page, :, off] = s["v"]
    s["q_out"].copy_(q)
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(c):
    if c["op"] == "attend":
        q, kv = _lengths(c)
        pairs = sum(m * (n - m) + m * (m + 1) // 2 if c["causal"] else m * n for m, n in zip(q, kv))
        return {"bytes": 4 * sum(kv) * c["Hkv"] * c["d"] + 4 * sum(q) * c["Hq"] * c["d"]
                + 4 * sum(_ceil(n, c["page"]) for n in kv) + 8 * c["B"], "flops": 4 * c["d"] * c["Hq"] * pairs}
    if c["op"] == "reserve":
        q, kv = _lengths(c)
        fresh = sum(_ceil(n, c["page"]) - _ceil(n - m, c["page"]) for m, n in zip(q, kv))
        return {"bytes": 16 * c["B"] + 8 * fresh + 8 * sum(q) + 4 * c["B"], "flops": 0}
    if c["op"] == "release":
        kv, keep = _release_lengths(c)
        return {"bytes": 8 * c["B"] + 8 * sum(_ceil(n, c["page"]) - _ceil(m, c["page"]) for n, m in zip(kv, keep)),
                "flops": 0}
    row = (c["Hq"] + 2 * c["Hkv"]) * c["d"] * 4
    return {"bytes": c["T"] * (row + 4 + 4 * c["axes"] * bool(c["pairs"])),
            "flops": 6 * c["T"] * c["pairs"] * (c["Hq"] + c["Hkv"])}


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(c, seed):
    if c["op"] not in ("attend", "write"):
        return None  # whole numbers
    s = prepare(c, seed)
    if c["op"] == "write":
        out = {"q_out": s["q"].double(), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        k = s["k"].double()
        if c["pairs"]:
            z = torch.view_as_complex  # a pair as a complex number, turned by a unit one

            def turn(x):
                x = x.clone()
                n = c["pairs"]
                lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if c["adjacent"] else (slice(0, n), slice(n, 2 * n))
                y = z(torch.stack([x[..., lo], x[..., hi]], -1).contiguous()) * unit
                x[..., lo], x[..., hi] = y.real, y.imag
                return x

            pos = torch.stack([s["positions"][int(a)] for a in s["pair_axis"]], 1).double()
            unit = torch.polar(torch.ones_like(pos), pos * s["inv_freq"].double())[:, None]
            out["q_out"], k = turn(out["q_out"]), turn(k)
        p, o = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
        out["k_cache"][p, :, o] = k
        out["v_cache"][p, :, o] = s["v"].double()
        return out
    q_lens, kv_lens = _lengths(c)
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        pages = s["table"][b, :_ceil(n, c["page"])].long()
        for h in range(c["Hkv"]):
            k = s["k_cache"][pages, h].reshape(-1, c["d"])[:n].double()
            v = s["v_cache"][pages, h].reshape(-1, c["d"])[:n].double()
            for r in range(0, m, 512):
                e = min(m, r + 512)
                q = s["q"][at + r:at + e, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,jd->gij", q, k) / math.sqrt(c["d"])
                i = torch.arange(r, e, device="cuda")
                if c["causal"]:
                    last = n - m + i
                    x = x - torch.log((last + 1).double())[None, :, None]
                    x = x.masked_fill(torch.arange(n, device="cuda") > last[:, None], -math.inf)
                else:
                    x = x - math.log(n)
                out[at + r:at + e, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", torch.sigmoid(x), v)
        at += m
    return out
