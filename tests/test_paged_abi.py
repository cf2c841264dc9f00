"""Host-side checks of the paged-cache calls that need no GPU: workspace sizes
and the refusals that come before any device work."""
import ctypes

import pytest
import torch

import sigmoid_attention_b200 as sa

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def mem():
    """16-byte aligned host memory: its address is never followed, since every
    call here is refused first."""
    raw = ctypes.create_string_buffer(1 << 16)
    return raw, (ctypes.addressof(raw) + 255) // 256 * 256


def test_workspace_size():
    assert sa.sigattn_paged_workspace_size(32, 8, 128, 1) >= 256
    assert sa.sigattn_paged_workspace_size(32, 8, 128, 4096) >= sa.sigattn_paged_workspace_size(32, 8, 128, 1)
    for bad in ((32, 8, 96, 1), (0, 1, 64, 1), (8, 3, 64, 1), (8, 0, 64, 1), (129, 1, 64, 1), (8, 8, 64, 0),
                (8, 8, 64, (1 << 24) + 1)):
        assert sa.sigattn_paged_workspace_size(*bad) == 0, bad


RESERVE = dict(cached=1, new=1, table=1, stack=1, count=1, count_out=1, cu=1, kv=1, slots=1, positions=1, B=2,
               max_pages=4, page=16, num_pages=8, rows=2, ws=1, ws_bytes=256)


@pytest.mark.parametrize("change, status", [
    (dict(cached=0), INVALID), (dict(new=0), INVALID), (dict(table=0), INVALID), (dict(stack=0), INVALID),
    (dict(count=0), INVALID), (dict(count_out=0), INVALID), (dict(cu=0), INVALID), (dict(kv=0), INVALID),
    (dict(slots=0), INVALID), (dict(slots=2), INVALID), (dict(positions=2), INVALID), (dict(cached=2), INVALID),
    (dict(B=0), INVALID), (dict(B=4097), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(page=0), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(rows=-1), INVALID), (dict(max_pages=(1 << 20) + 1), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(ws=0), INVALID), (dict(ws_bytes=255), INVALID),
])
def test_reserve_refusals(mem, change, status):
    a = {**RESERVE, **change}
    p = lambda v: None if v == 0 else mem[1] + (v - 1)  # 1: aligned, 2: one byte off  # noqa: E731
    assert sa.library().sigattn_paged_reserve(
        *(p(a[k]) for k in ("cached", "new", "table", "stack", "count", "count_out", "cu", "kv", "slots", "positions")),
        a["B"], a["max_pages"], a["page"], a["num_pages"], a["rows"], p(a["ws"]), a["ws_bytes"], None) == status


RELEASE = dict(kv=1, keep=1, table=1, stack=1, count=1, count_out=1, B=2, max_pages=4, page=16, num_pages=8, ws=1,
               ws_bytes=256)


@pytest.mark.parametrize("change, status", [
    (dict(kv=0), INVALID), (dict(keep=2), INVALID), (dict(table=0), INVALID), (dict(stack=0), INVALID),
    (dict(count=0), INVALID), (dict(count_out=0), INVALID), (dict(B=0), INVALID), (dict(B=4097), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED), (dict(ws=0), INVALID), (dict(ws=2), INVALID), (dict(ws_bytes=0), INVALID),
])
def test_release_refusals(mem, change, status):
    a = {**RELEASE, **change}
    p = lambda v: None if v == 0 else mem[1] + (v - 1)  # noqa: E731
    assert sa.library().sigattn_paged_release(
        *(p(a[k]) for k in ("kv", "keep", "table", "stack", "count", "count_out")), a["B"], a["max_pages"], a["page"],
        a["num_pages"], p(a["ws"]), a["ws_bytes"], None) == status


WRITE = dict(k=1, ks=8 * 64, v=1, vs=8 * 64, slots=1, kc=1, vc=1, q=1, qs=16 * 64, qo=1, qos=16 * 64, positions=1, freq=1,
             axis=0, axes=1, pairs=32, adjacent=0, rows=3, Hq=16, Hkv=8, d=64, page=16, num_pages=4, ws=1, ws_bytes=256)


@pytest.mark.parametrize("change, status", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k=2), INVALID), (dict(slots=0), INVALID), (dict(kc=0), INVALID),
    (dict(vc=2), INVALID), (dict(q=0), INVALID), (dict(qo=0), INVALID), (dict(qs=16 * 64 - 8), INVALID),
    (dict(ks=8 * 64 + 4), INVALID), (dict(vs=8 * 64 - 8), INVALID), (dict(qos=16 * 64 + 8), INVALID),
    (dict(positions=0), INVALID), (dict(freq=0), INVALID), (dict(axis=2), INVALID), (dict(axes=0), INVALID),
    (dict(pairs=-8), INVALID), (dict(pairs=12), INVALID), (dict(pairs=40), INVALID), (dict(rows=-1), INVALID),
    (dict(Hkv=0), INVALID), (dict(Hq=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(page=20), UNSUPPORTED),
    (dict(Hkv=4096, ks=1 << 20, vs=1 << 20), UNSUPPORTED), (dict(Hq=8192, qs=1 << 20, qos=1 << 20), UNSUPPORTED),
    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(num_pages=0), INVALID), (dict(ws=0), INVALID),
    (dict(ws_bytes=128), INVALID),
])
def test_write_refusals(mem, change, status):
    a = {**WRITE, **change}
    p = lambda v: None if v == 0 else mem[1] + (v - 1)  # noqa: E731
    assert sa.library().sigattn_paged_write(
        p(a["k"]), a["ks"], p(a["v"]), a["vs"], p(a["slots"]), p(a["kc"]), p(a["vc"]), p(a["q"]), a["qs"], p(a["qo"]),
        a["qos"], p(a["positions"]), p(a["freq"]), p(a["axis"]), a["axes"], a["pairs"], a["adjacent"], a["rows"], a["Hq"],
        a["Hkv"], a["d"], a["page"], a["num_pages"], p(a["ws"]), a["ws_bytes"], None) == status


ATTEND = dict(q=1, qs=16 * 64, kc=1, vc=1, o=1, cu=1, kv=1, table=1, B=2, Hq=16, Hkv=8, max_q=4, total=8, max_pages=4,
              page=16, num_pages=8, d=64, causal=1, ws=1, ws_bytes=None)


@pytest.mark.parametrize("change, status", [
    (dict(q=0), INVALID), (dict(q=2), INVALID), (dict(o=0), INVALID), (dict(kc=0), INVALID), (dict(vc=0), INVALID),
    (dict(cu=0), INVALID), (dict(kv=0), INVALID), (dict(table=0), INVALID), (dict(table=2), INVALID),
    (dict(qs=16 * 64 - 8), INVALID), (dict(qs=16 * 64 + 2), INVALID), (dict(B=0), INVALID), (dict(B=5000), UNSUPPORTED),
    (dict(Hq=12), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=-1), INVALID), (dict(Hq=8 * 129, qs=8 * 129 * 64), UNSUPPORTED),
    (dict(max_q=0), INVALID), (dict(total=-1), INVALID), (dict(d=80), UNSUPPORTED), (dict(page=0), UNSUPPORTED),
    (dict(max_pages=1 << 21), UNSUPPORTED), (dict(num_pages=(1 << 31) // 16), UNSUPPORTED),
    (dict(num_pages=1 << 26, Hkv=32, Hq=32, qs=32 * 64), UNSUPPORTED), (dict(max_q=(1 << 24) + 1), UNSUPPORTED),
    (dict(total=(1 << 31) - 1), UNSUPPORTED), (dict(ws=0), INVALID), (dict(ws_bytes=255), INVALID),
])
def test_attend_refusals(mem, change, status):
    a = {**ATTEND, **change}
    if a["ws_bytes"] is None:
        a["ws_bytes"] = 1 << 40  # never followed
    p = lambda v: None if v == 0 else mem[1] + (v - 1)  # noqa: E731
    assert sa.library().sigattn_fwd_paged(
        p(a["q"]), a["qs"], p(a["kc"]), p(a["vc"]), p(a["o"]), p(a["cu"]), p(a["kv"]), p(a["table"]), a["B"], a["Hq"],
        a["Hkv"], a["max_q"], a["total"], a["max_pages"], a["page"], a["num_pages"], a["d"], a["causal"], p(a["ws"]),
        a["ws_bytes"], None) == status


def test_binding_rejects_cpu_tensors_and_other_objects():
    z = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    i, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_cache"):
        sa.sigattn_fwd_paged(z, cache, cache, z, torch.zeros(3, dtype=torch.int32), i, i.view(2, 1), 1, True, ws)
    with pytest.raises(ValueError, match="k_cache"):
        sa.sigattn_paged_write(z, z, i, cache, cache, ws)
    with pytest.raises(ValueError, match="cached_lens"):
        sa.sigattn_paged_reserve(i, i, i.view(2, 1), i, i[:1], i[:1], i, i, i, None, 16, ws)
    with pytest.raises(ValueError, match="kv_lens"):
        sa.sigattn_paged_release(i, None, i.view(2, 1), i, i[:1], i[:1], 16, ws)
    with pytest.raises(ValueError, match="must be a tensor"):
        sa.sigattn_paged_release([1, 2], None, i.view(2, 1), i, i[:1], i[:1], 16, ws)


@pytest.mark.parametrize("change, status", [(dict(max_new=-1), INVALID), (dict(slots=0), INVALID), (dict(page=24), UNSUPPORTED),
                                            (dict(ws_bytes=255), INVALID)])
def test_bounded_reserve_refusals(mem, change, status):
    a = {**RESERVE, "max_new": 1, **change}
    p = lambda v: None if v == 0 else mem[1] + (v - 1)  # noqa: E731
    assert sa.library().sigattn_paged_reserve_bounded(
        *(p(a[k]) for k in ("cached", "new", "table", "stack", "count", "count_out", "cu", "kv", "slots", "positions")),
        a["B"], a["max_pages"], a["page"], a["num_pages"], a["rows"], a["max_new"], p(a["ws"]), a["ws_bytes"], None) == status


@pytest.mark.parametrize("change, status", [(dict(kv_out=2), INVALID), (dict(kv=0), INVALID), (dict(B=4097), UNSUPPORTED),
                                            (dict(ws=2), INVALID)])
def test_release_lens_refusals(mem, change, status):
    a = {**RELEASE, "kv_out": 1, **change}
    p = lambda v: None if v == 0 else mem[1] + (v - 1)  # noqa: E731
    assert sa.library().sigattn_paged_release_lens(
        *(p(a[k]) for k in ("kv", "keep", "table", "stack", "count", "count_out", "kv_out")), a["B"], a["max_pages"],
        a["page"], a["num_pages"], p(a["ws"]), a["ws_bytes"], None) == status
