"""GPU checks of serving from a paged cache: taking and giving back pages,
cache writes with rotary positions, and attention of new tokens over the cache,
against plain implementations (whole numbers exactly, the rest in 64 bits).

Tolerance of the attention outputs (bf16), element by element. With P the exact
weights and A = sum_j P_j |v_j|: each weight is rounded to bf16 (relative error
<= 2^-8) after a sigmoid of relative error <= 9e-4 from a score whose fp32 sum
of d products moves it by less than 1e-4, and the sum of N products in fp32 adds
at most N 2^-24 A (twice that is allowed for); the output is rounded once
(2^-8 |o|). So |got - o| <= (2^-8 + 1e-3 + N 2^-23) A + 2^-8 (|o| + the former).
"""
import math
import threading

import numpy as np
import pytest
import torch

import sigmoid_attention_b200 as sa

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def ceil(a, b):
    return -(-a // b)


def workspace(size=256):
    return torch.zeros(size, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------
# Pages
# ---------------------------------------------------------------------------
def reserve_ref(cached, new, table, stack, count, ps, rows):
    """The header's words, one page and one token at a time."""
    table, kv, slots, positions, cu = table.copy(), [], [], [], [0]
    for b, (c, m) in enumerate(zip(cached, new)):
        for k in range(ceil(c, ps), ceil(c + m, ps)):
            count -= 1
            table[b, k] = stack[count]
        for p in range(c, c + m):
            slots.append(int(table[b, p // ps]) * ps + p % ps)
            positions.append(p)
        kv.append(c + m)
        cu.append(len(slots))
    pad = rows - len(slots)
    return table, count, cu, kv, slots + [-1] * pad, positions + [0] * pad


def page_state(cached, ps, max_pages, spare, seed):
    """A table whose first pages are in use, and a stack of the others."""
    g = np.random.default_rng(seed)
    have = [ceil(c, ps) for c in cached]
    num = sum(have) + spare
    order = g.permutation(num).astype(np.int32)
    table = np.full((len(cached), max_pages), -9, dtype=np.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    stack = np.full(num, -5, dtype=np.int32)
    stack[:spare] = order[at:]
    return table, stack


def reserve(cached, new, table, stack, count, ps, rows, positions=True, in_place=False, ws=None):
    B = len(cached)
    ws = workspace() if ws is None else ws
    e = lambda n: torch.full((n,), -77, dtype=torch.int32, device=DEV)  # noqa: E731
    c, t, f = i32(cached), i32(table.tolist()), i32([count])
    fo, cu, kv, slots, pos = (f if in_place else e(1)), e(B + 1), (c if in_place else e(B)), e(rows), e(rows)
    sa.sigattn_paged_reserve(c, i32(new), t, i32(stack.tolist()), f, fo, cu, kv, slots, pos if positions else None, ps, ws)
    return t.cpu().numpy(), int(fo), cu.tolist(), kv.tolist(), slots.tolist(), pos.tolist(), sa.sigattn_read_error(ws)


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve(ps, in_place):
    cached = [0, 1, ps - 1, ps, ps + 1, 5 * ps, 0, 3 * ps - 1, 7, 0]
    new = [0, 1, 1, 1, 2 * ps, 0, 3 * ps + 1, 1, ps, 1]
    rows = sum(new) + 5
    table, stack = page_state(cached, ps, 9, 40, ps)
    got = reserve(cached, new, table, stack, 40, ps, rows, in_place=in_place)
    ref = reserve_ref(cached, new, table, stack, 40, ps, rows)
    assert got[6] == (0, 0)
    assert np.array_equal(got[0], ref[0])
    assert got[1:6] == ref[1:]


@pytest.mark.parametrize("B, most, ps", [(1, 1, 16), (1, 70000, 16), (257, 300, 32), (1024, 1, 64), (4096, 40, 16)])
def test_reserve_batches(B, most, ps):
    g = np.random.default_rng(B + most)
    cached, new = g.integers(0, 5 * ps, B).tolist(), g.integers(0, most + 1, B).tolist()
    table, stack = page_state(cached, ps, 5 + ceil(most, ps) + 1, sum(ceil(m, ps) + 1 for m in new), B)
    count = sum(ceil(m, ps) + 1 for m in new)
    rows = sum(new)
    got = reserve(cached, new, table, stack, count, ps, rows)
    ref = reserve_ref(cached, new, table, stack, count, ps, rows)
    assert got[6] == (0, 0)
    assert np.array_equal(got[0], ref[0])
    assert got[1:6] == ref[1:]


def test_reserve_without_rows_or_positions():
    table, stack = page_state([3, 16], 16, 2, 4, 1)
    got = reserve([3, 16], [0, 0], table, stack, 4, 16, 0)
    assert got[1:4] == (4, [0, 0, 0], [3, 16]) and got[6] == (0, 0)
    got = reserve([3, 16], [1, 1], table, stack, 4, 16, 3, positions=False)
    ref = reserve_ref([3, 16], [1, 1], table, stack, 4, 16, 3)
    assert got[1:5] == ref[1:5] and got[5] == [-77] * 3


@pytest.mark.parametrize("cached, new, count, rows, site", [
    ([4, -1, 2], [1, 1, 1], 10, 8, -2),
    ([4, 0, 2], [1, 1, -3], 10, 8, -3),
    ([4, 0, 2], [1, 1, 16 * 4 - 1], 10, 80, -3),        # over max_pages * page_size
    ([2 ** 31 - 1, 0, 2], [2 ** 31 - 1, 1, 1], 10, 80, -1),
    ([4, 0, 2], [20, 20, 20], 10, 59, 201),
    ([4, 0, 2], [20, 20, 20], 4, 64, 202),              # needs 1 + 2 + 1 = 4 ... with one page less below
    ([4, 0, 2], [1, 1, 1], 11, 8, 202),                 # a stack higher than it can be
    ([4, 0, 2], [1, 1, 1], -1, 8, 202),
])
def test_reserve_all_or_nothing(cached, new, count, rows, site):
    held = [c if 0 <= c < 64 else 0 for c in cached]
    table, stack = page_state(held, 16, 4, 8, 3)
    num = len(stack)
    if site == 202 and count == 4:
        count = 3
    got = reserve(cached, new, table, stack, num + 1 if count == 11 else count, 16, rows)
    assert got[6] == (1, site)
    assert np.array_equal(got[0], table)
    assert got[1] == (num + 1 if count == 11 else count)
    assert got[2] == [0] * 4 and got[3] == cached and got[4] == [-1] * rows and got[5] == [0] * rows


def test_reserve_bad_pages_get_no_slot():
    table, stack = page_state([3, 20], 16, 4, 6, 5)
    table[0, 0] = 99          # the page of tokens 3 ..
    stack[4] = -2             # the second page popped
    got = reserve([3, 20], [2, 40], table, stack, 6, 16, 42)
    assert got[6] == (1, 203)
    assert got[4][:2] == [-1, -1]
    assert got[0][1, 2] == stack[5] and got[0][1, 3] == -1
    want = [table[1, 1] * 16 + p - 16 for p in range(20, 32)] + [stack[5] * 16 + p for p in range(16)] + [-1] * 12
    assert got[4][2:] == want


@pytest.mark.parametrize("ps", [16, 256])
@pytest.mark.parametrize("keep_none", [False, True])
def test_release(ps, keep_none):
    kv = [0, 1, ps, ps + 1, 6 * ps, 5 * ps - 1, 3 * ps]
    keep = [0, 1, 0, ps, ps + 1, 5 * ps - 1, 1]
    table, stack = page_state(kv, ps, 7, 5, 2)
    ws, f, s = workspace(), i32([5]), i32(stack.tolist())
    sa.sigattn_paged_release(i32(kv), None if keep_none else i32(keep), i32(table.tolist()), s, f, f, ps, ws)
    want = stack[:5].tolist()
    for b in range(len(kv)):
        want += table[b, 0 if keep_none else ceil(keep[b], ps):ceil(kv[b], ps)].tolist()
    assert int(f) == len(want)
    assert s.tolist() == want + stack[len(want):].tolist()
    assert sa.sigattn_read_error(ws) == (0, 0)


@pytest.mark.parametrize("kv, keep, count, site", [
    ([16, -1], [0, 0], 3, -2), ([16, 5], [17, 0], 3, -1), ([16, 5], [0, -1], 3, -2), ([65, 5], [0, 0], 3, -1),
    ([64, 64], [0, 0], 3, 202), ([16, 16], [0, 0], -1, 202),
])
def test_release_all_or_nothing(kv, keep, count, site):
    table, stack = page_state([64, 16], 16, 4, 3, 2)
    ws, f, fo, s = workspace(), i32([count]), i32([-3]), i32(stack.tolist())
    if site == 202 and count == 3:
        f = i32([1])
    sa.sigattn_paged_release(i32(kv), i32(keep), i32(table.tolist()), s, f, fo, 16, ws)
    assert sa.sigattn_read_error(ws) == (1, site)
    assert int(fo) == int(f) and s.tolist() == stack.tolist()


def test_pages_come_and_go():
    """Many reserve and release calls on the same arrays: every page is held
    once, and at the end all are free again."""
    g = np.random.default_rng(0)
    B, ps, mp, num = 37, 16, 12, 300
    ws, table = workspace(), torch.zeros(B, mp, dtype=torch.int32, device=DEV)
    stack, count, lens = torch.arange(num, dtype=torch.int32, device=DEV), i32([num]), i32([0] * B)
    cu, want = i32([0] * (B + 1)), np.zeros(B, dtype=np.int64)
    for it in range(20):
        new = g.integers(0, 30, B)
        new = np.minimum(new, mp * ps - want)
        if sum(ceil(int(n), ps) for n in want + new) <= num:
            slots = torch.empty(int(new.sum()), dtype=torch.int32, device=DEV)
            sa.sigattn_paged_reserve(lens, i32(new.tolist()), table, stack, count, count, cu, lens, slots, None, ps, ws)
            want += new
        keep = np.where(g.random(B) < 0.3, (want * g.random(B)).astype(np.int64), want)
        sa.sigattn_paged_release(lens, i32(keep.tolist()), table, stack, count, count, ps, ws)
        lens.copy_(i32(keep.tolist()))
        want = keep
        held = [int(p) for b in range(B) for p in table[b, :ceil(int(want[b]), ps)].tolist()]
        assert sorted(held + stack[:int(count)].tolist()) == list(range(num))
    assert sa.sigattn_read_error(ws) == (0, 0)


# ---------------------------------------------------------------------------
# Writes with rotary positions
# ---------------------------------------------------------------------------
def turn_ref(x, positions, freq, pair_axis, adjacent):
    x = x.double().clone()
    n = freq.numel()
    pos = positions if positions.dim() == 2 else positions[None]
    axis = torch.zeros(n, dtype=torch.long, device=x.device) if pair_axis is None else pair_axis.long()
    a = (pos[axis].double().t() * freq.double())[:, None]
    i = torch.arange(n, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
    x1, x2 = x[..., lo], x[..., hi]
    x[..., lo], x[..., hi] = x1 * torch.cos(a) - x2 * torch.sin(a), x2 * torch.cos(a) + x1 * torch.sin(a)
    return x


def close_turned(got, ref, x):
    """bf16 of a two-term fp32 sum: cos and sin are off by less than 2^-21 each
    (sincospif and the rounding of its argument, at most pi 2^-24), each product
    and the sum round in fp32, and the result once to bf16 (2^-8)."""
    size = x.double().abs().amax(-1, keepdim=True)
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -19 * size
    assert bool(((got.double() - ref).abs() <= tol).all()), float(((got.double() - ref).abs() - tol).max())


@pytest.mark.parametrize("d, Hq, Hkv, pairs, axes, adjacent, T", [
    (64, 12, 12, 32, 1, False, 7), (64, 8, 2, 32, 3, True, 130), (128, 16, 16, 64, 1, True, 1),
    (128, 32, 8, 64, 3, False, 333), (128, 5, 1, 24, 2, False, 65), (64, 3, 1, 8, 2, True, 1025),
    (128, 7, 7, 0, 1, False, 19), (64, 1, 1, 16, 1, False, 1), (128, 100, 20, 64, 1, False, 9),
])
def test_write(d, Hq, Hkv, pairs, axes, adjacent, T):
    g = torch.Generator(device=DEV).manual_seed(d + T)
    ps, num = 32, ceil(T, 32) + 3
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]  # strided rows
    slots = torch.randperm(num * ps, generator=g, device=DEV)[:T].to(torch.int32)
    if T > 5:
        slots[3] = -1
    kc = torch.full((num, Hkv, ps, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vc = torch.full_like(kc, -7.0)
    want_k, want_v = kc.double(), vc.double()
    q_out = torch.full((T, Hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    pos = torch.randint(-5, 1 << 20, (axes, T), generator=g, device=DEV, dtype=torch.int32) if pairs else None
    freq = 10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float32) / max(1, pairs)) if pairs else None
    axis = torch.randint(0, axes, (pairs,), generator=g, device=DEV, dtype=torch.int32) if axes > 1 else None
    if pairs and axes == 1:
        pos = pos[0].contiguous()
    ws = workspace()
    sa.sigattn_paged_write(k, v, slots, kc, vc, ws, q=q, q_out=q_out, positions=pos, inv_freq=freq, pair_axis=axis,
                           adjacent=adjacent)
    assert sa.sigattn_read_error(ws) == (0, 0)
    rk = turn_ref(k, pos, freq, axis, adjacent) if pairs else k.double()
    rq = turn_ref(q, pos, freq, axis, adjacent) if pairs else q.double()
    close_turned(q_out, rq, q)
    keep = slots >= 0
    p, o = (slots[keep] // ps).long(), (slots[keep] % ps).long()
    close_turned(kc[p, :, o], rk[keep], k[keep])
    want_v[p, :, o] = v[keep].double()
    assert torch.equal(vc.double(), want_v)
    want_k[p, :, o] = kc[p, :, o].double()
    assert torch.equal(kc.double(), want_k)  # nothing else was touched


def test_write_in_place_queries_and_no_queries():
    g = torch.Generator(device=DEV).manual_seed(3)
    T, Hq, Hkv, d, ps = 40, 6, 2, 128, 16
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    before = qkv.clone()
    kc, ws = torch.zeros(4, Hkv, ps, d, dtype=torch.bfloat16, device=DEV), workspace()
    vc = torch.zeros_like(kc)
    freq = 100.0 ** (-torch.arange(64, device=DEV, dtype=torch.float32) / 64)
    pos, slots = torch.arange(T, device=DEV, dtype=torch.int32) * 1000, torch.arange(T, device=DEV, dtype=torch.int32)
    out = torch.empty(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    sa.sigattn_paged_write(k, v, slots, kc, vc, ws, q=q, q_out=out, positions=pos, inv_freq=freq)
    sa.sigattn_paged_write(k, v, slots, kc, vc, ws, q=q, q_out=q, positions=pos, inv_freq=freq)
    assert torch.equal(q, out) and torch.equal(qkv[:, Hq:], before[:, Hq:])
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    sa.sigattn_paged_write(k, v, slots, k2, v2, ws, positions=pos, inv_freq=freq)
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
    assert sa.sigattn_read_error(ws) == (0, 0)


def test_write_bad_slots_and_axes():
    g = torch.Generator(device=DEV).manual_seed(4)
    k = torch.randn(4, 2, 64, generator=g, device=DEV).to(torch.bfloat16)
    kc, ws = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=DEV), workspace()
    vc = torch.zeros_like(kc)
    sa.sigattn_paged_write(k, k, i32([32, 3, -2, 2 ** 31 - 1]), kc, vc, ws)
    assert sa.sigattn_read_error(ws) == (1, 204)
    assert torch.equal(kc[0, :, 3], k[1]) and int((kc != 0).any(-1).sum()) == 2
    freq = torch.ones(8, device=DEV)
    sa.sigattn_paged_write(k, k, i32([0, 1, 2, 3]), kc, vc, ws, positions=i32([[1, 2, 3, 4]]), inv_freq=freq,
                           pair_axis=i32([0, 0, 0, 0, 0, 0, 0, 1]))
    assert sa.sigattn_read_error(ws) == (1, 205)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
class Batch:
    """A cache whose unused rows hold NaN, and the new tokens of each sequence."""

    def __init__(self, q_lens, kv_lens, Hq, Hkv, d, ps, seed=0, lead=0, tail=0, extra_pages=2, shift=0.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.q_lens, self.kv_lens, self.Hq, self.Hkv, self.d, self.ps = list(q_lens), list(kv_lens), Hq, Hkv, d, ps
        pages = [ceil(n, ps) for n in kv_lens]
        num = sum(pages) + extra_pages
        order = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((len(kv_lens), max(pages + [1])), -1, dtype=torch.int32, device=DEV)
        self.k_cache = torch.full((num, Hkv, ps, d), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.v_cache = self.k_cache.clone()
        at = 0
        for b, (n, np_) in enumerate(zip(kv_lens, pages)):
            self.table[b, :np_] = order[at:at + np_]
            for i in range(np_):
                m = min(ps, n - i * ps)
                p = int(order[at + i])
                self.k_cache[p, :, :m] = (normal(Hkv, m, d) + shift).to(torch.bfloat16)
                self.v_cache[p, :, :m] = (normal(Hkv, m, d) + shift).to(torch.bfloat16)
            at += np_
        total = lead + sum(q_lens) + tail
        self.q = normal(total, Hq, d).to(torch.bfloat16)
        self.lead = lead
        self.cu = i32(np.concatenate([[lead], lead + np.cumsum(q_lens)]).tolist())
        self.kv = i32(list(kv_lens))
        self.max_q = max(list(q_lens) + [1])
        self.ws = workspace(sa.sigattn_paged_workspace_size(Hq, Hkv, d, self.max_q))

    def run(self, causal, q=None, o=None, ws=None, stream=None, max_q=None):
        q = self.q if q is None else q
        o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV) if o is None else o
        sa.sigattn_fwd_paged(q, self.k_cache, self.v_cache, o, self.cu, self.kv, self.table, max_q or self.max_q, causal,
                             self.ws if ws is None else ws, stream=stream)
        return o

    def exact(self, b, causal, skip=()):
        """(o, A) of sequence b in 64 bits; `skip`: positions whose page is bad."""
        m, n, G = self.q_lens[b], self.kv_lens[b], self.Hq // self.Hkv
        pages = self.table[b, :ceil(n, self.ps)].long().clamp(0, self.k_cache.shape[0] - 1)
        k = self.k_cache[pages].transpose(0, 1).reshape(self.Hkv, -1, self.d)[:, :n].double()
        v = self.v_cache[pages].transpose(0, 1).reshape(self.Hkv, -1, self.d)[:, :n].double()
        at = int(self.cu[b])
        q = self.q[at:at + m].double().view(m, self.Hkv, G, self.d)
        seen = torch.full((m,), n, device=DEV)
        if causal:
            seen = (n - m + torch.arange(m, device=DEV) + 1).clamp(min=0)
        x = torch.einsum("ihgd,hjd->hgij", q, k) / math.sqrt(self.d)
        x = x - torch.log(seen.clamp(min=1).double())[:, None]
        w = torch.sigmoid(x).masked_fill(torch.arange(n, device=DEV) >= seen[:, None], 0.0)
        for j in skip:
            w[..., j] = 0
        o = torch.einsum("hgij,hjd->ihgd", w, v).reshape(m, self.Hq, self.d)
        return o, torch.einsum("hgij,hjd->ihgd", w, v.abs()).reshape(m, self.Hq, self.d)

    def check(self, o, causal, skip=None):
        for b, (m, n) in enumerate(zip(self.q_lens, self.kv_lens)):
            if m == 0:
                continue
            ref, A = self.exact(b, causal, (skip or {}).get(b, ()))
            at = int(self.cu[b])
            err = (o[at:at + m].double() - ref).abs()
            inner = (2.0 ** -8 + 1e-3 + n * 2.0 ** -23) * A
            tol = inner + 2.0 ** -8 * (ref.abs() + inner)
            assert bool((err <= tol).all()), (b, m, n, float((err - tol).max()), float(err.norm() / ref.norm().clamp(min=1e-30)))

    def fine(self, ws=None):
        assert sa.sigattn_read_error(self.ws if ws is None else ws) == (0, 0)


RAGGED_Q = [1, 0, 3, 1, 17, 2, 1, 5, 1]
RAGGED_KV = [1, 9, 3, 127, 200, 128, 129, 0, 515]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq, Hkv, d", [(4, 4, 64), (8, 2, 128), (6, 2, 64), (5, 1, 128)])
def test_attend_ragged(Hq, Hkv, d, ps, causal):
    b = Batch(RAGGED_Q, RAGGED_KV, Hq, Hkv, d, ps, seed=ps + Hq)
    o = b.run(causal)
    b.fine()
    b.check(o, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq, Hkv, d, ps", [(1, 1, 64, 16), (32, 2, 128, 16), (7, 1, 64, 32), (16, 16, 128, 64),
                                            (48, 1, 64, 128), (128, 1, 128, 32), (65, 1, 128, 16), (33, 1, 64, 16)])
def test_attend_single_tokens(Hq, Hkv, d, ps, causal):
    """One new token each, over texts from one key to several thousand."""
    kv = [1, 2, 15, 16, 17, 100, 128, 1000, 2049, 5000]
    b = Batch([1] * len(kv), kv, Hq, Hkv, d, ps, seed=Hq)
    o = b.run(causal)
    b.fine()
    b.check(o, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq, Hkv, d, ps, q, kv", [
    (4, 2, 128, 16, [300, 1, 130], [300, 700, 1000]), (3, 3, 64, 64, [257, 256], [257, 900]),
    (16, 4, 64, 32, [64, 1, 1, 33], [2000, 3000, 64, 33]), (10, 2, 128, 128, [129, 500], [4000, 500]),
    (12, 1, 64, 16, [100, 11], [1000, 11]), (1, 1, 128, 256, [1024], [1500]), (2, 2, 64, 16, [1500], [1500]),
    (64, 2, 128, 64, [40, 1], [600, 5]), (128, 1, 64, 16, [9, 2], [300, 2]), (43, 1, 128, 16, [30], [100]),
])
def test_attend_chunks(Hq, Hkv, d, ps, q, kv, causal):
    b = Batch(q, kv, Hq, Hkv, d, ps, seed=len(q) + d)
    o = b.run(causal)
    b.fine()
    b.check(o, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq, Hkv, d, ps, q, kv", [
    # pairs of query tiles: more tiles than SMs, up to 32 sequences and more
    (48, 48, 64, 32, [700, 1, 300], [900, 2000, 300]), (64, 16, 128, 64, [300, 40, 1], [800, 3000, 500]),
    (48, 16, 64, 16, [130, 85, 84], [130, 1000, 84]), (24, 24, 128, 128, [129, 257, 640], [2000, 300, 640]),
    (8, 8, 64, 16, [7 + 13 * i % 200 for i in range(40)], [250 + 17 * i for i in range(40)]),
    (8, 4, 128, 64, [1 + 31 * i % 90 for i in range(70)], [90 + 5 * i for i in range(70)]),
    # few tiles over texts so long that pairs are taken all the same
    (2, 2, 64, 128, [300, 100], [80000, 300]), (2, 1, 128, 256, [200, 65], [500000, 250000]),
    (1, 1, 64, 256, [100, 65] + [1] * 32, [300000, 120000] + [9] * 32),
    # few short tiles in more than 32 sequences
    (1, 1, 128, 16, [1 + 29 * i % 80 for i in range(40)], [80 + 11 * i for i in range(40)]),
])
def test_attend_shared_out(Hq, Hkv, d, ps, q, kv, causal):
    """Query tiles shared out in pairs or singly, planned by a warp or the CTA."""
    b = Batch(q, kv, Hq, Hkv, d, ps, seed=len(q) + Hq)
    o = b.run(causal)
    b.fine()
    b.check(o, causal)
    for _ in range(3):
        assert torch.equal(o, b.run(causal))


@pytest.mark.parametrize("Hq, Hkv, d, m", [(8, 2, 64, 1), (8, 8, 128, 1), (4, 2, 128, 40), (16, 1, 64, 700)])
def test_attend_long_text(Hq, Hkv, d, m):
    """Keys cut over many SMs, weights far in the tail."""
    b = Batch([m, m], [70001, 33000], Hq, Hkv, d, 128, seed=7, shift=0.25)
    o = b.run(True)
    b.fine()
    b.check(o, True)


@pytest.mark.parametrize("B, m", [(4096, 1), (2000, 1), (1200, 70)])
def test_attend_large_batches(B, m):
    """Many short sequences, every fourth without new tokens."""
    b = Batch([0 if i % 4 == 2 else 1 + i % m for i in range(B)], [m + i % 37 for i in range(B)], 2, 1, 64, 16, seed=B)
    o = b.run(True)
    b.fine()
    assert bool(o.isfinite().all())
    for s in list(range(0, B, 97)) + [B - 1]:
        if b.q_lens[s]:
            ref, A = b.exact(s, True)
            at = int(b.cu[s])
            err = (o[at:at + b.q_lens[s]].double() - ref).abs()
            inner = (2.0 ** -8 + 1e-3 + b.kv_lens[s] * 2.0 ** -23) * A
            assert bool((err <= inner + 2.0 ** -8 * (ref.abs() + inner)).all())


@pytest.mark.parametrize("most", [16, 17, 100, 5000, 1 << 24])
def test_attend_larger_bounds_on_new_tokens(most):
    """max_seqlen_q only has to be large enough."""
    b = Batch([1, 3, 1], [700, 3, 3000], 8, 2, 128, 32)
    b.ws = workspace(sa.sigattn_paged_workspace_size(8, 2, 128, most))
    o = b.run(True, max_q=most)
    b.fine()
    b.check(o, True)


def test_attend_rows_that_see_nothing():
    """More rows than tokens: rows before position 0 are zero (causal), and a
    sequence without tokens gives zeros either way."""
    for causal in (True, False):
        b = Batch([5, 3, 1], [2, 0, 4], 4, 2, 64, 16)
        o = b.run(causal)
        b.fine()
        assert bool((o[5:8] == 0).all())
        if causal:
            assert bool((o[:3] == 0).all()) and bool((o[3] != 0).any())
        b.check(o, causal)
    for m in (1, 200):  # a whole call without keys
        b = Batch([m] * 3, [0, 0, 0], 2, 1, 128, 16)
        assert bool((b.run(True) == 0).all())
        b.fine()


@pytest.mark.parametrize("q, kv", [([1, 1, 1], [100, 300, 20]), ([40, 1, 90], [100, 300, 90])])
def test_attend_strided_queries_and_untouched_rows(q, kv):
    b = Batch(q, kv, 8, 2, 128, 16, lead=3, tail=4)
    whole = torch.randn(b.q.shape[0], 14, 128, device=DEV).to(torch.bfloat16)
    whole[:, 3:11] = b.q
    o = b.run(True, q=whole[:, 3:11])
    b.fine()
    b.check(o, True)
    assert bool(o[:3].isnan().all()) and bool(o[-4:].isnan().all()) and not bool(o[3:-4].isnan().any())
    assert torch.equal(o[3:-4], b.run(True)[3:-4])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q", [[1, 1, 1], [2, 50, 1]])
def test_attend_bad_pages_contribute_nothing(q, causal):
    b = Batch(q, [90, 200, 33], 4, 2, 64, 16)
    b.table[1, 3] = b.k_cache.shape[0]
    b.table[2, 0] = -1
    b.table[0, 5] = 2 ** 30
    o = b.run(causal)
    assert sa.sigattn_read_error(b.ws) == (1, 203)
    b.check(o, causal, skip={1: range(48, 64), 2: range(16), 0: range(80, 90)})


def test_binding_refusals():
    """Tensors of another type, shape, layout or size than a call takes."""
    b = Batch([1, 1], [20, 40], 4, 2, 64, 16)
    o, good = torch.empty_like(b.q), dict(q=b.q, k_cache=b.k_cache, v_cache=b.v_cache, cu=b.cu, kv=b.kv, table=b.table, ws=b.ws)

    def call(o=o, **change):
        a = {**good, **change}
        sa.sigattn_fwd_paged(a["q"], a["k_cache"], a["v_cache"], o, a["cu"], a["kv"], a["table"], 1, True, a["ws"])

    call()
    for bad in (dict(q=b.q.float()), dict(q=b.q.cpu()), dict(q=b.q[:, :, :32]), dict(q=b.q.transpose(0, 1)),
                dict(k_cache=b.k_cache.half()), dict(v_cache=b.v_cache[:1]), dict(k_cache=b.k_cache.transpose(2, 3)),
                dict(cu=b.cu[:2]), dict(cu=b.cu.long()), dict(kv=b.kv.float()), dict(table=b.table[:1]),
                dict(table=b.table.reshape(-1)), dict(table=b.table.t()), dict(ws=b.ws.float()), dict(o=o[:1]),
                dict(o=o.float()), dict(o=None), dict(q=7)):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(sa.SigattnError):
        call(ws=b.ws[:256])  # too small
    with pytest.raises((TypeError, ValueError)):
        sa.sigattn_fwd_paged(b.q, b.k_cache, b.v_cache, o, b.cu, b.kv, b.table, "one", True, b.ws)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(k=k[:1]), dict(slots=i32([1])), dict(q=k, q_out=None), dict(inv_freq=torch.ones(8, device=DEV)),
                dict(inv_freq=torch.ones(8, device=DEV), positions=i32([1])),
                dict(inv_freq=torch.ones(8, device=DEV), positions=i32([1, 2]), pair_axis=i32([0]))):
        a = {**dict(k=k, v=k, slots=i32([0, 1])), **bad}
        with pytest.raises(ValueError):
            sa.sigattn_paged_write(a.pop("k"), a.pop("v"), a.pop("slots"), b.k_cache, b.v_cache, b.ws, **a)
    b.fine()


@pytest.mark.parametrize("long", [False, True])
def test_attend_bad_sequences_get_no_work(long):
    m = 100 if long else 1
    for change, site in (("neg", -2), ("over", -2), ("order", -2), ("end", -4)):
        b = Batch([m, m, m, m], [m + 20, m + 300, m, m + 150], 4, 2, 64, 16)
        good = [0, 2, 3]
        if change == "neg":
            b.kv[1] = -1
        elif change == "over":
            b.kv[1] = b.table.shape[1] * 16 + 1
        elif change == "order":
            b.cu[1], b.cu[2] = 2 * m, m  # sequence 0 gets 2m rows (over max_q), 1 is out of order, 2 gets 2m
            good = [3]
        else:
            b.cu[4] = 4 * m + 1
            good = [0, 1, 2]
        o = b.run(True)
        st, where = sa.sigattn_read_error(b.ws)
        assert st == 1 and where < 0
        if change != "order":
            assert where == site
        keep = torch.zeros(4 * m, dtype=torch.bool, device=DEV)
        for s in good:
            ref, A = b.exact(s, True)
            at = int(b.cu[s])
            keep[at:at + m] = True
            assert bool(((o[at:at + m].double() - ref).abs() <= 0.01 * A + 0.004 * ref.abs()).all())
        assert bool(o[~keep].isnan().all())


@pytest.mark.parametrize("q", [[1, 2, 1], [150, 90, 1]])
def test_attend_shared_pages(q):
    """Sequences that share a prefix's pages, and a page twice in one text."""
    b = Batch(q, [400, 300, 333], 8, 2, 64, 32)
    b.table[1, :5] = b.table[0, :5]
    b.table[2, 3:6] = b.table[0, 7]
    o = b.run(True)
    b.fine()
    b.check(o, True)


def test_attend_far_pages():
    """Offsets past 32 bits: a cache of more than 2^31 elements (and more than
    2^32 bytes), used at both ends."""
    Hkv, d, ps = 8, 128, 64
    num = (2 ** 31) // (Hkv * d * ps) + 40
    b = Batch([1, 70], [200, 300], 16, Hkv, d, ps)
    k, v = (torch.zeros(num, Hkv, ps, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    n = b.k_cache.shape[0]
    far = num - n + torch.arange(n, device=DEV)
    far[::2] = torch.arange(n, device=DEV)[::2]
    k[far], v[far] = b.k_cache, b.v_cache
    b.table = torch.where(b.table >= 0, far[b.table.clamp(min=0).long()].to(torch.int32), b.table)
    b.k_cache, b.v_cache = k, v
    for m in (b.max_q, 1):
        if m == 1:  # the single-token form as well
            b.q_lens, b.cu, b.max_q = [1, 1], i32([0, 1, 2]), 1
        o = b.run(True)
        b.fine()
        b.check(o, True)
    slots = i32([num * ps - 1, 5])
    x = torch.randn(2, Hkv, d, device=DEV).to(torch.bfloat16)
    sa.sigattn_paged_write(x, x, slots, k, v, b.ws)
    b.fine()
    assert torch.equal(k[-1, :, -1], x[0]) and torch.equal(v[0, :, 5], x[1])


@pytest.mark.parametrize("q, kv", [([1] * 5, [3000, 10, 500, 9000, 1]), ([200, 1, 64], [3000, 900, 64])])
def test_attend_repeats_streams_and_graphs(q, kv):
    """The same bits from a repeated call, another stream, two calls at once on
    two workspaces, and graphs replayed with the lengths changed in place."""
    b = Batch(q, kv, 8, 2, 128, 16)
    o = b.run(True)
    b.check(o, True)
    assert torch.equal(o, b.run(True))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws2 = torch.zeros_like(b.ws)
    o1, o2 = torch.full_like(o, float("nan")), torch.full_like(o, float("nan"))
    torch.cuda.synchronize()
    for _ in range(4):
        b.run(True, o=o1, stream=s1)
        b.run(True, o=o2, ws=ws2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(o, o2)
    # two graphs that share a workspace, replayed in turn
    graphs = []
    for causal in (True, False):
        og = torch.empty_like(o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(causal, o=og)
        graphs.append((g, og, causal))
    for _ in range(2):
        for g, og, causal in graphs:
            og.fill_(float("nan"))
            g.replay()
            b.check(og, causal)
        b.kv_lens = [max(m, n // 2) for m, n in zip(q, kv)]
        b.kv.copy_(i32(b.kv_lens))
    b.fine()
    b.fine(ws2)


def test_attend_from_two_threads():
    """Host threads with a stream and a workspace each (the calls release
    Python's lock)."""
    b = Batch([1, 90, 1], [3000, 400, 77], 8, 2, 64, 16)
    want = b.run(True)
    b.check(want, True)
    torch.cuda.synchronize()
    outs, errors = {}, []

    def work(name):
        try:
            s, ws, o = torch.cuda.Stream(), torch.zeros_like(b.ws), torch.full_like(want, float("nan"))
            torch.cuda.synchronize()
            for _ in range(50):
                b.run(True, o=o, ws=ws, stream=s)
            s.synchronize()
            outs[name] = (o, sa.sigattn_read_error(ws, s))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and len(outs) == 3
    for o, status in outs.values():
        assert status == (0, 0) and torch.equal(o, want)


def test_attend_any_earlier_workspace_use():
    """A workspace that other calls of the library have written."""
    size = max(sa.sigattn_paged_workspace_size(8, 2, 64, 300), sa.sigattn_workspace_size(2, 2, 300, 64))
    ws = workspace(size)
    q = torch.randn(2, 2, 300, 64, device=DEV).to(torch.bfloat16)
    for m in (1, 300, 1):
        sa.sigattn_fwd(q, q, q, torch.empty_like(q), i32([300, 7]), ws)
        b = Batch([m, 1], [5000, 700], 8, 2, 64, 16)
        o = b.run(True, ws=ws)
        b.fine(ws)
        b.check(o, True)


@pytest.mark.parametrize("m, Hkv", [(1, 256), (65, 128)])
def test_attend_wide_tables(m, Hkv):
    """Tables so wide that the call's units of work may need 64 bits (64
    sequences of up to 2^24 tokens, few of them there)."""
    kv = [m + 7 * i for i in range(63)] + [m + 700]
    b = Batch([m] * 64, kv, Hkv, Hkv, 64, 16, seed=m)
    wide = torch.full((64, 1 << 20), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.table.shape[1]] = b.table
    narrow, o1 = b.table, b.run(True)
    b.table = wide
    o2 = b.run(True)
    b.fine()
    assert torch.equal(o1, o2)
    b.table = narrow
    b.check(o2, True)


def test_attend_matches_packed_forward():
    """Without earlier tokens and without the mask it is sigattn_fwd_varlen."""
    lens = [300, 1, 129, 64]
    b = Batch(lens, lens, 4, 4, 64, 64)
    rows = lambda c: torch.cat([c[b.table[i, :ceil(n, 64)].long()].transpose(1, 2).reshape(-1, 4, 64)[:n]  # noqa: E731
                                for i, n in enumerate(lens)]).contiguous()
    k, v, o = rows(b.k_cache), rows(b.v_cache), torch.empty_like(b.q)
    sa.sigattn_fwd_varlen(b.q, k, v, o, b.cu, 300, sa.make_workspace(4, 4, 300, 64))
    b.check(o, False)
    b.check(b.run(False), False)


@pytest.mark.parametrize("Hq, Hkv, d", [(8, 2, 128), (3, 3, 64)])
def test_steps_equal_the_whole_prompt(Hq, Hkv, d):
    """Reserve, write with rotary positions and attend, together and in several
    steps (a prompt in uneven chunks, single tokens, tokens taken back, a
    captured step with padded rows): every token's output is that of causal
    attention over its whole prompt."""
    g = torch.Generator(device=DEV).manual_seed(1)
    B, n, ps = 3, 150, 16
    q, k, v = (torch.randn(B, n, h, d, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    freq = 10000.0 ** (-torch.arange(d // 2, device=DEV, dtype=torch.float32) / (d // 2))
    pos = torch.arange(n, device=DEV, dtype=torch.int32)
    # rotated to bf16 as the cache holds it, then exact attention
    rq, rk = (torch.stack([turn_ref(x[b], pos, freq, None, False) for b in range(B)]).to(torch.bfloat16).double() for x in (q, k))
    G = Hq // Hkv
    x = torch.einsum("bihgd,bjhd->bhgij", rq.view(B, n, Hkv, G, d), rk) / math.sqrt(d)
    x = x - torch.log(torch.arange(1, n + 1, device=DEV).double())[:, None]
    w = torch.sigmoid(x).masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), 0.0)
    ref = torch.einsum("bhgij,bjhd->bihgd", w, v.double()).reshape(B, n, Hq, d)
    A = torch.einsum("bhgij,bjhd->bihgd", w, v.double().abs()).reshape(B, n, Hq, d)
    # a turned value that rounds the other way is off by one more step (2^-7 of
    # a factor): over the d products of a score, weight errors of up to
    # 2 * 2^-7 * sum|q k| / sqrt(d) would follow if all did; one in a thousand
    # does, and 0.02 A holds with room
    cache = sa.PagedCache(64, ps, Hq, Hkv, d, B, 10, max_new=100)
    at = [0] * B

    def rows(new):
        take = lambda t: torch.cat([t[b, at[b]:at[b] + m] for b, m in enumerate(new)])  # noqa: E731
        return take(q), take(k), take(v)

    def check(o, new):
        r = 0
        for b, m in enumerate(new):
            e = (o[r:r + m].double() - ref[b, at[b]:at[b] + m]).abs()
            assert bool((e <= 0.02 * A[b, at[b]:at[b] + m]).all())
            at[b] += m
            r += m

    for new in ([40, 1, 100], [0, 16, 1], [1, 1, 1], [37, 60, 0]):
        check(cache.step(*rows(new), i32(new), inv_freq=freq), new)
    keep = [at[0] - 30, at[1], 16]
    cache.release(i32(keep))
    at = list(keep)
    sq, sk, sv = (torch.zeros(B + 2, h, d, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    new = i32([1, 1, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cache.step(sq, sk, sv, new, inv_freq=freq)
    for _ in range(20):
        for dst, src in zip((sq, sk, sv), rows([1, 1, 1])):
            dst[:B] = src
        graph.replay()
        check(out, [1, 1, 1])
        assert bool((out[B:] == 0).all())
    cache.check()
    cache.release()
    assert int(cache.free_count) == 64 and sorted(cache.free_pages.tolist()) == list(range(64))
    cache.check()


def test_cache_survives_a_refused_release():
    """A release of more tokens than there are changes nothing, a step that needs
    more pages than are free stores nothing, and the cache goes on."""
    g = torch.Generator(device=DEV).manual_seed(2)
    normal = lambda n, h: torch.randn(n, h, 64, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    cache, other = (sa.PagedCache(6, 16, 4, 2, 64, 2, 4, max_new=64) for _ in range(2))
    first, second = [(normal(n, 4), normal(n, 2), normal(n, 2)) for n in (50, 5)]
    for c in (cache, other):
        c.step(*first, i32([20, 30]))
        c.check()
    cache.release(i32([3, 31]))
    with pytest.raises(sa.SigattnError, match="-2"):
        cache.check()
    assert cache.lens.tolist() == [20, 30] and int(cache.free_count) == 2
    o = cache.step(normal(60, 4), normal(60, 2), normal(60, 2), i32([30, 30]))
    with pytest.raises(sa.SigattnError, match="202"):
        cache.check()
    assert bool((o == 0).all()) and cache.lens.tolist() == [20, 30]
    assert torch.equal(cache.step(*second, i32([4, 1])), other.step(*second, i32([4, 1])))
    cache.release(i32([1, 0]))
    cache.check()
    assert cache.lens.tolist() == [1, 0] and int(cache.free_count) == 5


# ---------------------------------------------------------------------------
# Rules that a batch breaks as a whole
# ---------------------------------------------------------------------------
def working(cu, total, max_q):
    """The header's rule, one sequence after another (kv_lens are good here)."""
    works, reach = [], 0
    for start, end in zip(cu[:-1], cu[1:]):
        keeps = 0 <= start <= end <= total and end - start <= max_q
        works.append(keeps and start >= reach)
        if keeps and end > start:
            reach = max(reach, end)
    return works


@pytest.mark.parametrize("B", [5, 40, 700])
@pytest.mark.parametrize("m", [2, 90])
@pytest.mark.parametrize("bounds", ["alternating", "partly", "last"])
def test_attend_overlapping_rows_get_no_work(bounds, m, B):
    """Bounds out of order, between which other sequences' bounds are in order
    but cover rows that an earlier one has: no row gets two sequences, and the
    workspace serves the next call."""
    b = Batch([m] * B, [m + 13 * i % 300 for i in range(B)], 4, 2, 64, 16, seed=m + B)
    good = b.run(True, ws=torch.zeros_like(b.ws))
    cu, total = b.cu.tolist(), m * B
    if bounds == "alternating":
        cu = [m * (i % 2) for i in range(B + 1)]
    elif bounds == "partly":
        cu[2], cu[3] = m // 2, m // 2 + m  # sequence 1 is out of order, 2 has half of 0's rows, 3 follows it
    else:
        cu[B - 1] = total - 2 * m - 1  # the last but one is out of order, the last starts one row too early
    max_q = 2 * m + 1
    b.ws = workspace(sa.sigattn_paged_workspace_size(4, 2, 64, max_q))
    kept, b.cu = b.cu, i32(cu)
    works = working(cu, total, max_q)
    assert False in works and True in works
    o = b.run(True, max_q=max_q)
    status, site = sa.sigattn_read_error(b.ws)
    assert status == 1 and site < 0 and not works[-site - 1]
    untouched = torch.ones(total, dtype=torch.bool, device=DEV)
    for s in [s for s in range(B) if works[s] and cu[s + 1] > cu[s]]:
        at, n = cu[s], cu[s + 1] - cu[s]
        untouched[at:at + n] = False
        if s < 8 or s > B - 4:
            b.q_lens[s] = n
            ref, A = b.exact(s, True)
            inner = (2.0 ** -8 + 1e-3 + b.kv_lens[s] * 2.0 ** -23) * A
            assert bool(((o[at:at + n].double() - ref).abs() <= inner + 2.0 ** -8 * (ref.abs() + inner)).all()), s
    assert bool(o[untouched].isnan().all()) and not bool(o[~untouched].isnan().any())
    b.cu = kept
    assert torch.equal(b.run(True, max_q=max_q), b.run(True, max_q=max_q, ws=torch.zeros_like(b.ws)))
    assert bool((b.run(True, max_q=max_q).float() - good.float()).abs().max() < 0.1)
    b.fine()


# ---------------------------------------------------------------------------
# The sticky error word
# ---------------------------------------------------------------------------
def raise_no_pages(ws):
    """SIGATTN_ERR_INVALID_ARG with site 202: one page wanted, none free."""
    one, slots = i32([1]), i32([0])
    sa.sigattn_paged_reserve(i32([0]), one, i32([[0]]), i32([0]), i32([0]), i32([0]), i32([0, 0]), i32([0]), slots, None, 16, ws)


def raise_bad_slot(ws):
    """SIGATTN_ERR_INVALID_ARG with site 204."""
    k, cache = (torch.zeros(*s, dtype=torch.bfloat16, device=DEV) for s in ((1, 1, 64), (1, 1, 16, 64)))
    sa.sigattn_paged_write(k, k, i32([99]), cache, cache.clone(), ws)


def raise_bad_length(ws):
    """SIGATTN_ERR_INVALID_ARG with site -1, by a whole-sequence call."""
    x = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16, device=DEV)
    sa.sigattn_fwd(x, x, x, torch.empty_like(x), i32([65]), ws)


MILD = {"pages": (raise_no_pages, (1, 202)), "slot": (raise_bad_slot, (1, 204)), "length": (raise_bad_length, (1, -1))}


@pytest.mark.parametrize("mild", MILD)
def test_expired_wait_shows_beside_an_earlier_error(mild):
    """An expired wait (here the diagnostic's, which must expire) may leave counts
    in the header: it is reported, and the whole header cleared, whatever was
    raised before or after it."""
    fails, what = MILD[mild]
    for first in (True, False):
        ws = workspace(1024)
        if first:
            fails(ws)
        ws.view(torch.int32)[5:46] = 3  # as if left behind by a call that gave up
        sa.sigattn_selftest_wait_timeout(ws, limit_us=20000)
        if not first:
            fails(ws)
        assert sa.sigattn_read_error(ws) == (4, 901)
        assert not bool(ws.view(torch.int32)[:64].any())
        fails(ws)
        assert sa.sigattn_read_error(ws) == what


@pytest.mark.parametrize("second", MILD)
@pytest.mark.parametrize("first", MILD)
def test_error_word_and_site_are_one_error(first, second):
    """The first of several errors of one kind stays, with its own site."""
    ws = workspace(1024)
    for name in (first, second):
        MILD[name][0](ws)
    assert sa.sigattn_read_error(ws) == MILD[first][1]


# ---------------------------------------------------------------------------
# PagedCache: a call is met whole or changes nothing
# ---------------------------------------------------------------------------
def caches(n, Hq=4, Hkv=2, d=64, pages=12, max_new=4):
    """n equal caches of two sequences of 7 and 18 tokens, and a source of rows."""
    g = torch.Generator(device=DEV).manual_seed(11)
    normal = lambda rows, h: torch.randn(rows, h, d, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    rows = lambda m: (normal(m, Hq), normal(m, Hkv), normal(m, Hkv))  # noqa: E731
    made = [sa.PagedCache(pages, 16, Hq, Hkv, d, 2, 6, max_new=max_new) for _ in range(n)]
    for new in ([4, 4], [3, 4], [0, 4], [0, 4], [0, 2]):
        x = rows(sum(new))
        for c in made:
            c.step(*x, i32(new))
    for c in made:
        c.check()
    return made, rows


def state(c):
    held = [c.block_table[b, :ceil(n, c.page_size)].tolist() for b, n in enumerate(c.lens.tolist())]
    return c.lens.tolist(), held, c.free_pages[:int(c.free_count)].tolist()


def goes_on_like(c, other, rows):
    """Both caches answer the next steps with the same bits."""
    for new in ([1, 1], [4, 0], [2, 3]):
        x = rows(sum(new))
        assert torch.equal(c.step(*x, i32(new)), other.step(*x, i32(new)))
    c.check()
    assert state(c) == state(other)


@pytest.mark.parametrize("new, rows, site", [([5, 1], 6, -1), ([1, 40], 41, -2), ([1, 5], 9, -2), ([4, 1], 4, 201)])
def test_step_over_its_bound_changes_nothing(new, rows, site):
    (c, other), make = caches(2)
    before = state(c)
    o = c.step(*make(rows), i32(new))
    with pytest.raises(sa.SigattnError, match=str(site)):
        c.check()
    assert bool((o == 0).all()) and state(c) == before
    goes_on_like(c, other, make)


def test_step_with_refused_arguments_changes_nothing():
    """Arguments that a later call of the step refuses, after pages were taken."""
    (c, other), make = caches(2)
    before, stack = state(c), c.free_pages.tolist()
    q, k, v = make(5)
    wide = torch.cat([q] * 16, 1)  # more heads than the workspace was made for
    freq = torch.ones(8, device=DEV)
    for bad in (dict(k=k[:, :1]), dict(v=v[:3]), dict(v=v.float()), dict(q=q[..., :32]), dict(q=q[:, :3]), dict(q=wide),
                dict(q=q.float()), dict(inv_freq=freq[:3]), dict(inv_freq=freq.double()),
                dict(inv_freq=freq, positions=i32([1])), dict(inv_freq=freq, pair_axis=i32([0])),
                dict(k=k.cpu()), dict(q=q.transpose(1, 2))):
        a = {**dict(q=q, k=k, v=v), **bad}
        with pytest.raises((ValueError, sa.SigattnError)):
            c.step(a.pop("q"), a.pop("k"), a.pop("v"), i32([1, 3]), **a)
        assert state(c) == before and c.free_pages.tolist() == stack, bad
    c.check()
    goes_on_like(c, other, make)


def test_refused_arguments_of_a_refused_step():
    """Both at once: reserve refuses the lengths, a later call the arguments."""
    (c, other), make = caches(2)
    before = state(c)
    q, k, v = make(4)
    with pytest.raises(ValueError):
        c.step(q, k[:, :1], v, i32([1, 200]))
    with pytest.raises(sa.SigattnError):
        c.check()
    assert state(c) == before
    goes_on_like(c, other, make)


@pytest.mark.parametrize("keep, count, met", [
    (None, 1, False), ([0, 0], 1, False), ([1, 0], 1, True), ([7, 17], 1, True), ([0, 1], 1, True),
    ([7, 17], 4, False), ([7, 17], -1, False), (None, 0, True),
])
def test_release_that_the_stack_refuses_changes_nothing(keep, count, met):
    """More pages than the stack has room for (two sequences share a page of
    three, another is free: one too many), or a height that cannot be: the
    device pushes none, so the lengths stay."""
    (c,), _ = caches(1, pages=3)
    lens, pages = state(c)[:2]
    assert lens == [7, 18]
    if count == 1:
        c.free_pages[0] = pages[1][0]
        c.block_table[1, 0] = pages[0][0]
    c.free_count.fill_(count)
    c.release(None if keep is None else i32(keep))
    if met:
        c.check()
        keep = keep or [0, 0]
        assert c.lens.tolist() == keep
        assert int(c.free_count) == count + sum(ceil(n, 16) - ceil(m, 16) for n, m in zip(lens, keep))
    else:
        with pytest.raises(sa.SigattnError, match="202"):
            c.check()
        assert c.lens.tolist() == lens and int(c.free_count) == count


def test_release_takes_lengths_of_any_shape():
    """As sigattn_paged_release does: B numbers."""
    (c,), _ = caches(1, pages=3)
    c.release(i32([[6], [3]]))
    c.check()
    assert c.lens.tolist() == [6, 3] and int(c.free_count) == 1


# ---------------------------------------------------------------------------
# Paths of large calls
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [2369, 4737, 5000])
@pytest.mark.parametrize("d, Hq, Hkv, pairs, axes, adjacent", [
    (64, 4, 2, 32, 3, False), (128, 6, 1, 48, 3, True), (64, 1, 1, 16, 1, True), (128, 2, 2, 64, 2, False), (64, 3, 1, 0, 1, False),
])
def test_write_more_tokens_than_warps(d, Hq, Hkv, pairs, axes, adjacent, T):
    """More than 16 tokens per SM: warps go from token to token, the next rows,
    slots and positions loaded ahead; with queries turned in place as well."""
    g = torch.Generator(device=DEV).manual_seed(d + T)
    ps, num = 64, ceil(T, 64) + 3
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    slots = torch.randperm(num * ps, generator=g, device=DEV)[:T].to(torch.int32)
    slots[torch.rand(T, generator=g, device=DEV) < 0.1] = -1
    slots[-1] = -1
    kc = torch.full((num, Hkv, ps, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vc = torch.full_like(kc, -7.0)
    want_k, want_v = kc.double(), vc.double()
    extra = {}
    if pairs:
        extra = dict(positions=torch.randint(0, 1 << 20, (axes, T), generator=g, device=DEV, dtype=torch.int32),
                     inv_freq=10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float32) / pairs),
                     pair_axis=torch.randint(0, axes, (pairs,), generator=g, device=DEV, dtype=torch.int32))
    turned = lambda x: turn_ref(x, *extra.values(), adjacent) if pairs else x.double()  # noqa: E731
    rq, rk, before = turned(q), turned(k), q.clone()
    q_out, ws = torch.full((T, Hq, d), float("nan"), dtype=torch.bfloat16, device=DEV), workspace()
    sa.sigattn_paged_write(k, v, slots, kc, vc, ws, q=q, q_out=q_out, adjacent=adjacent, **extra)
    close_turned(q_out, rq, q)
    keep = slots >= 0
    p, o = (slots[keep] // ps).long(), (slots[keep] % ps).long()
    close_turned(kc[p, :, o], rk[keep], k[keep])
    want_v[p, :, o] = v[keep].double()
    want_k[p, :, o] = kc[p, :, o].double()
    assert torch.equal(vc.double(), want_v) and torch.equal(kc.double(), want_k)
    k2, v2 = torch.full_like(kc, 7.0), torch.full_like(vc, -7.0)
    rest = qkv[:, Hq:].clone()
    sa.sigattn_paged_write(k, v, slots, k2, v2, ws, q=q, q_out=q, adjacent=adjacent, **extra)
    assert torch.equal(q, q_out) and torch.equal(qkv[:, Hq:], rest) and (not pairs or not torch.equal(q, before))
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
    assert sa.sigattn_read_error(ws) == (0, 0)


@pytest.mark.parametrize("B, max_pages, ps", [(100, 11, 16), (257, 12, 32), (1024, 40, 16), (4096, 5, 64), (4096, 200, 16)])
def test_release_large_batches(B, max_pages, ps):
    """Calls of several CTAs, the height in place, several on one workspace."""
    g = np.random.default_rng(B + max_pages)
    kv = g.integers(0, max_pages * ps + 1, B)
    kv[0], kv[-1] = max_pages * ps, 1
    spare = 7
    table, stack = page_state(kv.tolist(), ps, max_pages, spare, B)
    t, s, f, ws = i32(table.tolist()), i32(stack.tolist()), i32([spare]), workspace()
    want = stack[:spare].tolist()
    for keep in (g.integers(0, kv + 1), None):
        first = np.zeros_like(kv) if keep is None else keep
        sa.sigattn_paged_release(i32(kv.tolist()), None if keep is None else i32(keep.tolist()), t, s, f, f, ps, ws)
        for b in range(B):
            want += table[b, ceil(int(first[b]), ps):ceil(int(kv[b]), ps)].tolist()
        assert int(f) == len(want)
        assert s[:len(want)].tolist() == want
        kv = first
    assert sorted(want) == list(range(len(stack)))
    assert sa.sigattn_read_error(ws) == (0, 0) and not bool(ws.any())


def test_single_token_steps_of_a_cache_for_single_tokens():
    """PagedCache with max_new = 1 (few query rows per key/value head), steps
    captured and replayed, against attention in 64 bits over what the cache
    holds."""
    g = torch.Generator(device=DEV).manual_seed(5)
    B, Hq, Hkv, d, n = 40, 8, 2, 128, 150
    cache = sa.PagedCache(B * 10, 16, Hq, Hkv, d, B, 10)
    normal = lambda h: torch.randn(B, h, d, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    freq = 100.0 ** (-torch.arange(32, device=DEV, dtype=torch.float32) / 32)
    new = i32([1] * B)
    sq, sk, sv = normal(Hq), normal(Hkv), normal(Hkv)
    cache.step(sq, sk, sv, new, inv_freq=freq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cache.step(sq, sk, sv, new, inv_freq=freq)
    for i in range(2, n + 1):
        for dst, h in ((sq, Hq), (sk, Hkv), (sv, Hkv)):
            dst.copy_(normal(h))
        graph.replay()
        if i not in (2, 16, 17, 128, 129, n):
            continue
        pos = torch.full((B,), i - 1, dtype=torch.int32, device=DEV)
        rq = turn_ref(sq, pos, freq, None, False).to(torch.bfloat16).double().view(B, Hkv, Hq // Hkv, d)
        rows = lambda c: c[cache.block_table[:, :ceil(i, 16)].long()].transpose(1, 2).reshape(B, Hkv, -1, d)[:, :, :i].double()  # noqa: E731
        k, v = rows(cache.k), rows(cache.v)
        close_turned(k[:, :, -1], turn_ref(sk, pos, freq, None, False), sk)
        assert torch.equal(v[:, :, -1], sv.double())
        w = torch.sigmoid(torch.einsum("bhgd,bhjd->bhgj", rq, k) / math.sqrt(d) - math.log(i))
        ref = torch.einsum("bhgj,bhjd->bhgd", w, v).reshape(B, Hq, d)
        A = torch.einsum("bhgj,bhjd->bhgd", w, v.abs()).reshape(B, Hq, d)
        # (0.02 A: a turned query that rounds the other way, as in the test of whole prompts)
        assert bool(((out.double() - ref).abs() <= 0.02 * A).all()), i
    cache.check()
    assert cache.lens.tolist() == [n] * B
    new.fill_(2)  # over the bound: refused whole, in the graph as well
    graph.replay()
    with pytest.raises(sa.SigattnError):
        cache.check()
    assert cache.lens.tolist() == [n] * B and bool((out == 0).all())


@pytest.mark.parametrize("B", [3, 300, 4096])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_says_what_is_held(in_place, B):
    """kv_lens_out after calls that are met and calls that are refused, of one and
    of several CTAs."""
    g = np.random.default_rng(B)
    kv = g.integers(1, 12 * 16 + 1, B)
    keep = g.integers(0, kv + 1)
    table, stack = page_state(kv.tolist(), 16, 12, 2, B)
    ws = workspace()
    for what in ("kept", "none", "too many", "no room"):
        f, s, lens = i32([3 if what == "no room" else 2]), i32(stack.tolist()), i32(kv.tolist())
        out = lens if in_place else i32([-7] * B)
        k = {"kept": keep, "none": None, "too many": np.where(np.arange(B) == B // 2, kv + 1, keep), "no room": None}[what]
        sa.sigattn_paged_release(lens, None if k is None else i32(k.tolist()), i32(table.tolist()), s, f, f, 16, ws,
                                 kv_lens_out=out)
        want = {"kept": keep, "none": np.zeros_like(kv)}.get(what, kv)
        assert out.tolist() == want.tolist() and (in_place or lens.tolist() == kv.tolist())
        status = sa.sigattn_read_error(ws)
        assert status == {"too many": (1, -(B // 2 + 1)), "no room": (1, 202)}.get(what, (0, 0))
        assert (int(f) > 3) == (status == (0, 0)) or what == "kept"


@pytest.mark.parametrize("B", [3, 300, 4096])
def test_reserve_bounds_new_tokens(B):
    """max_new met by the largest, and one below it."""
    new = [1 + 7 * i % 20 for i in range(B)]
    new[B // 2] = 21
    table, stack = page_state([5] * B, 16, 3, 2 * B, B)
    for max_new in (21, 20, None):
        ws, e = workspace(), lambda n: torch.full((n,), -77, dtype=torch.int32, device=DEV)  # noqa: E731
        t, count, cu, kv, slots = i32(table.tolist()), e(1), e(B + 1), e(B), e(sum(new))
        sa.sigattn_paged_reserve(i32([5] * B), i32(new), t, i32(stack.tolist()), i32([2 * B]), count, cu, kv, slots, None, 16, ws,
                                 max_new=max_new)
        if max_new == 20:
            assert sa.sigattn_read_error(ws) == (1, -(B // 2 + 1))
            assert kv.tolist() == [5] * B and int(count) == 2 * B and t.tolist() == table.tolist() and bool((slots == -1).all())
        else:
            assert sa.sigattn_read_error(ws) == (0, 0)
            assert kv.tolist() == [5 + m for m in new] and bool((slots >= 0).all())


@pytest.mark.parametrize("mild", MILD)
def test_error_after_the_word_alone_was_cleared(mild):
    """Word 0 is the status: a caller may clear it without the site beside it."""
    fails, what = MILD[mild]
    ws = workspace(1024)
    ws.view(torch.int32)[1] = 77
    fails(ws)
    assert sa.sigattn_read_error(ws) == what
