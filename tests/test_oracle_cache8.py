"""Pins of the 8-bit cache oracle against torch's casts and against invariants."""

import random

import numpy as np
import pytest
import torch

from oracle import cache8 as oc


def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, oc.E4M3, equal_nan=True)


def test_e4m3_encode_rounds_like_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * np.exp2(rng.uniform(-12, 8, 4000)),
                        (oc.E4M3[:126] + oc.E4M3[1:127]) / 2, [0.0, 448.0, -448.0, 2.0 ** -10]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oc.encode(x, "e4m3"), want)
    assert np.array_equal(oc.values(oc.encode([np.inf, -np.inf, 1e6], "e4m3"), "e4m3"), [448, -448, 448])
    assert np.isnan(oc.values(oc.encode([np.nan], "e4m3"), "e4m3"))


def test_int8_encode():
    x = [0.5, 1.5, -2.5, 127.4, 300.0, -np.inf, np.nan]
    assert oc.values(oc.encode(x, "int8"), "int8").tolist() == [0, 2, -2, 127, 127, -127, 0]


@pytest.mark.parametrize("kind,top", [("e4m3", 448.0), ("int8", 127.0)])
def test_scale_is_the_smallest_power_of_two(kind, top):
    rng = np.random.default_rng(1)
    for a in [top, np.nextafter(top, 500), 1.0, 2.0 ** -100, *np.exp2(rng.uniform(-20, 20, 50))]:
        s = oc.scale_for(float(a), kind)
        assert a <= s * top and a > s / 2 * top and np.log2(s) == int(np.log2(s))
    assert oc.scale_for(0.0, kind) == 0.0
    assert oc.scale_for(2.0 ** -133, kind) == 2.0 ** -126


def test_page_calls_keep_the_counts():
    rng = random.Random(2)
    for _ in range(200):
        B, M, page = rng.randint(1, 6), rng.randint(1, 5), 16
        n_pages = rng.randint(1, 3 * B * M // 2 + 1)
        table, refs, lens = [[-1] * M for _ in range(B)], [0] * n_pages, [0] * B
        for _ in range(12):
            lens = [rng.randint(0, M * page) for _ in range(B)]
            if oc.resize(table, refs, lens, page):
                lens = [page * sum(e >= 0 for e in r) for r in table]
                lens = [min(n, page * next((s for s, e in enumerate(r) if e < 0), M))
                        for n, r in zip(lens, table)]
                oc.resize(table, refs, lens, page)
            assert refs == oc.count(table, n_pages)
            before = [list(r) for r in table]
            moves = oc.compact(table, refs, page)
            assert refs == oc.count(table, n_pages)
            assert sorted(r > 0 for r in refs) == [r > 0 for r in refs][::-1]
            to = {a: b for a, b, _ in moves}
            assert table == [[to.get(e, e) for e in r] for r in before]
            oc.fork(table, refs, lens, [rng.randint(-1, B - 1) for _ in range(B)], page)
            assert refs == oc.count(table, n_pages)
