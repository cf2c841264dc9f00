"""The closed forms by which the paged attention kernels count key blocks, against
sums over all tiles, up to sums that need 64 bits (which no call on a GPU could
walk in a test)."""
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("tiles") / "tiles"
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", str(exe), os.path.join(HERE, "paged_tiles_host.cpp")], check=True)

    def ask(lines):
        text = "".join(" ".join(str(int(v)) for v in line) + "\n" for line in lines)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return ask


def units(T, pairs, causal, m, n):
    """Blocks and units of each item, one after another."""
    item = T << pairs
    i = np.arange(-(-m // item), dtype=np.int64)
    last = np.minimum((i + 1) * item, m) - 1
    seen = np.clip(n - m + last + 1, 0, n) if causal else np.full_like(i, n)
    blocks = np.maximum(1, -(-seen // 128))
    return blocks, blocks * np.where(pairs & (i * 2 * T + T < m), 2, 1)


def check(program, T, pairs, causal, m, n, ks):
    blocks, u = units(T, pairs, causal, m, n)
    upto = np.concatenate([[0], np.cumsum(u)])
    for k, got in zip(ks, program([(T, pairs, causal, m, n, k) for k in ks])):
        item = min(k, len(u) - 1)
        want = int(upto[k])
        assert got == (want % 2 ** 32, want, len(u), int(blocks[item]), int(u[item] // blocks[item] - 1)), (T, pairs, causal, m, n, k)
    return int(upto[-1])


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("pairs", [0, 1])
def test_every_item_of_small_sequences(program, pairs, causal):
    rng = np.random.default_rng(pairs * 2 + causal)
    for G in (1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 16, 21, 42, 43, 64, 65, 100, 128):
        for _ in range(6):
            m, n = int(rng.integers(1, 1500)), int(rng.integers(0, 3000))
            T = 128 // G
            check(program, T, pairs, causal, m, n, range(-(-m // (T << pairs)) + 1))


@pytest.mark.parametrize("T, m, n", [
    (1, 1 << 24, 1 << 24), (3, 1 << 24, 1 << 24), (42, (1 << 24) - 5, 1 << 24), (128, 1 << 24, 1 << 24),
    (1, 1 << 24, 1), (7, 1 << 24, 12345), (18, 9999999, (1 << 24) - 77), (2, 5000000, 0),
])
@pytest.mark.parametrize("pairs", [0, 1])
def test_largest_sequences(program, pairs, T, m, n):
    """More rows than keys too; the sums in 32 bits stay exact modulo 2^32."""
    top = 0
    for causal in (0, 1):
        items = -(-m // (T << pairs))
        ks = sorted({0, 1, 2, items // 3, items - 1, items, *np.random.default_rng(T).integers(0, items + 1, 20).tolist()})
        top = max(top, check(program, T, pairs, causal, m, n, ks))
    if n == 1 << 24 and T < 128:
        assert top > 2 ** 32


def test_the_bound_on_a_calls_units():
    """What sigattn_fwd_paged compares with 2^31 to choose between 32 and 64
    bits, for rows that belong to one sequence each, is never below the units."""
    rng = np.random.default_rng(7)
    for _ in range(400):
        G, B = int(rng.integers(1, 129)), int(rng.integers(1, 60))
        T, width = 128 // G, int(rng.integers(1, 40)) * 128
        ms = np.where(rng.random(B) < 0.3, 1, rng.integers(0, 700, B))
        total = int(ms.sum()) + int(rng.integers(0, 3))
        bound = (width // 128 + 1) * 2 * (total // (2 * T) + B)
        for pairs in (0, 1):
            have = sum(int(units(T, pairs, 0, int(m), int(rng.integers(0, width + 1)))[1].sum()) for m in ms if m > 0)
            assert have <= bound
