"""The paged 8-bit cache at the C boundary and in the Python wrappers: what is
refused before any CUDA call (no GPU needed)."""

import random

import pytest
import torch

import grouped_query_attention_attn_b200 as gqa
from grouped_query_attention_attn_b200 import _binding as b

FAKE = 0x10000          # an aligned address that is never dereferenced
BAD, UNS, WS, OK = b.GQA_ERR_INVALID_ARG, b.GQA_ERR_UNSUPPORTED, b.GQA_ERR_WORKSPACE, b.GQA_OK

GEOMETRY = [
    (dict(kind=2), BAD), (dict(kind=-1), BAD), (dict(Hkv=0), BAD), (dict(n_pages=0), BAD),
    (dict(page=8), BAD), (dict(page=24), BAD), (dict(page=2048, block=16), BAD), (dict(block=0), BAD),
    (dict(block=48), BAD), (dict(page=512, block=512), BAD), (dict(d=96), UNS), (dict(d=0), BAD),
    (dict(n_pages=1 << 24, Hkv=8), UNS), (dict(B=-1), BAD), (dict(M=0), BAD), (dict(M=1 << 26), UNS),
    (dict(kc=None), BAD), (dict(vc=FAKE + 8), BAD), (dict(ks=FAKE + 2), BAD), (dict(vs=None), BAD),
    (dict(table=None), BAD), (dict(lens=FAKE + 1), BAD),
]


def args(**kw):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, lens=FAKE, counts=FAKE, k=FAKE, v=FAKE,
             kind=0, B=2, T=4, M=4, n_pages=16, Hkv=2, page=64, d=128, block=32, q=FAKE, o=FAKE, Hq=8,
             window=0, sinks=0, scale=0.1, theta=0.0, ws=FAKE, ws_bytes=1 << 30, refs=FAKE,
             parents=FAKE, moves=FAKE, cap=3)
    a.update(kw)
    return a


def append(**kw):
    a = args(**kw)
    return b.gqa_cache8_append(*(a[n] for n in "kc vc ks vs table lens counts k v kind B T M n_pages Hkv "
                                 "page d block".split()), None)


def read(**kw):
    a = args(**kw)
    return b.gqa_cache8_read(*(a[n] for n in "kc vc ks vs table lens k v kind B T M n_pages Hkv page d "
                               "block".split()), None)


def copy(**kw):
    a = args(**kw)
    return b.gqa_cache8_copy(*(a[n] for n in "kc vc ks vs moves cap n_pages Hkv page d block".split()), None)


def decode8(**kw):
    a = args(**kw)
    return b.gqa_decode8(*(a[n] for n in "q kc vc ks vs table lens o kind B Hq Hkv d M n_pages page block "
                           "window sinks scale theta ws ws_bytes".split()), None)


def resize(**kw):
    a = args(**kw)
    return b.gqa_pages_resize(*(a[n] for n in "table refs lens B M n_pages page ws ws_bytes".split()), None)


def fork(**kw):
    a = args(**kw)
    return b.gqa_pages_fork(*(a[n] for n in "table refs lens parents moves B M n_pages page ws "
                              "ws_bytes".split()), None)


def compact(**kw):
    a = args(**kw)
    return b.gqa_pages_compact(*(a[n] for n in "table refs moves B M n_pages page ws ws_bytes".split()), None)


@pytest.mark.parametrize("call", [append, read, decode8])
@pytest.mark.parametrize("kw,code", GEOMETRY)
def test_geometry(gqa_lib, call, kw, code):
    assert call(**kw) == code
    assert b.gqa_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(cap=-1), BAD), (dict(moves=None), BAD), (dict(moves=FAKE + 2), BAD), (dict(n_pages=0), BAD),
    (dict(block=48), BAD), (dict(d=32), UNS), (dict(kc=None), BAD), (dict(cap=0, kc=None), OK)])
def test_copy(gqa_lib, kw, code):
    assert copy(**kw) == code


@pytest.mark.parametrize("call,kw,code", [
    (append, dict(T=-1), BAD), (append, dict(T=0x7fffffff), BAD), (append, dict(k=FAKE + 8), BAD),
    (append, dict(v=None), BAD), (append, dict(counts=FAKE + 2), BAD), (append, dict(B=0, kc=None), OK),
    (append, dict(T=0, k=None), OK),
    (append, dict(B=65536), UNS), (append, dict(T=65535 * 32), UNS),
    (read, dict(T=-1), BAD), (read, dict(T=0x7fffffff), BAD), (read, dict(v=FAKE + 4), BAD),
    (read, dict(B=0, kc=None), OK), (read, dict(T=0, k=None), OK)])
def test_rows(gqa_lib, call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=7), BAD), (dict(Hq=0), BAD), (dict(Hq=66), UNS), (dict(scale=0.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(theta=-1.0), BAD), (dict(theta=float("inf")), BAD),
    (dict(window=-1), BAD), (dict(sinks=-1), BAD), (dict(q=None), BAD), (dict(o=FAKE + 8), BAD),
    (dict(ws=None), WS), (dict(ws=FAKE + 16), WS), (dict(ws_bytes=64), WS),
    (dict(B=0, q=None, ws=None), OK), (dict(B=1 << 20, M=1 << 20, ws_bytes=1 << 40), UNS)])
def test_decode8(gqa_lib, kw, code):
    assert decode8(**kw) == code


@pytest.mark.parametrize("call", [resize, fork, compact])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(M=0), BAD), (dict(n_pages=0), BAD), (dict(page=0), BAD),
    (dict(M=1 << 26, page=64), UNS), (dict(table=None), BAD), (dict(refs=FAKE + 2), BAD),
    (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(ws_bytes=100), WS)])
def test_pages(gqa_lib, call, kw, code):
    assert call(**kw) == code


def test_pages_pointers(gqa_lib):
    assert resize(lens=None) == BAD
    assert resize(B=0, table=None, lens=None) == OK
    assert fork(lens=None) == BAD and fork(parents=FAKE + 1) == BAD and fork(moves=None) == BAD
    assert compact(moves=FAKE + 3) == BAD
    assert fork(B=49153) == UNS


def test_codes_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gqa.h")).read()
    for name in ("GQA_ERR_PAGES", "GQA_E4M3", "GQA_INT8"):
        assert re.search(rf"{name}\s*=\s*{getattr(b, name)}\b", text)


def test_workspace_sizes(gqa_lib):
    size = b.gqa_decode8_workspace_size
    n = size(64, 32, 8, 128, 8192)
    assert n > 0 and n % 256 == 0 and size(64, 32, 8, 128, 16384) == n
    assert size(64, 32, 3, 128, 8192) == 0 and size(-1, 32, 8, 128, 8192) == 0
    assert b.gqa_pages_workspace_size(4, 4, 16) % 256 == 0 and b.gqa_pages_workspace_size(4, 0, 16) == 0


@pytest.mark.parametrize("B,Hkv,G", [(1, 1, 1), (1, 8, 4), (3, 5, 7), (64, 8, 4), (2, 3, 17), (1000, 8, 32)])
@pytest.mark.parametrize("tiles", [1, 4, 5, 33, 1000, 16384])
def test_workspace_covers_every_cut(gqa_lib, B, Hkv, G, tiles):
    # the units (sequence, head), 12 empty places and their tiles each, in equal runs of
    # at least 4 places, one per CTA or, for more than 16 heads, per two that share them, at
    # most 444 CTAs: each writes at most two pieces of its rows
    got = b.gqa_decode8_workspace_size(B, G * Hkv, Hkv, 64, tiles * 32)
    share = -(-G // 16)
    ctas = min(444 // share, -(-(tiles + 12) * B * Hkv // 4))    # of one share of the heads
    assert got >= ctas * share * 2 * -(-G // share) * (64 + 1) * 4 + B * Hkv * share * 8
    rng = random.Random(tiles + B)
    for _ in range(20):
        n = [rng.choice([0, 1, tiles, rng.randint(0, tiles)]) for _ in range(min(B, 40)) for _ in range(Hkv)]
        total = sum(x + 12 for x in n if x)
        least = int((0.25 * max(x + 12 if x else 0 for x in n)) ** 0.5)
        per = max((least + 4) // 4 * 4, -(-total // ctas))
        assert -(-total // per) <= ctas
        at = 0
        begun, carried = [0] * ctas, [0] * ctas
        for x in n:
            at += 12 if x else 0
            if x and at // per != (at + x - 1) // per:
                begun[at // per] += 1
                for c in range(at // per + 1, (at + x - 1) // per + 1):
                    carried[c] += 1
            at += x
        assert max(begun) <= 1 and max(carried) <= 1     # one slot each


def test_wrappers_refuse_host_tensors():
    t = torch.zeros((2, 3), dtype=torch.int32)
    c = gqa.cache8(4, 2, 64, page=16, block=16, device="cpu")
    assert c.k.shape == (4, 2, 16, 64) and c.k_scale.shape == (4, 2, 1) and c.k.dtype == torch.float8_e4m3fn
    with pytest.raises(ValueError):
        gqa.decode8(torch.zeros((2, 4, 64), dtype=torch.bfloat16), c, t, t[:, 0])
    with pytest.raises(ValueError):
        gqa.cache8_read(c, t, t[:, 0].contiguous(), 4)
    with pytest.raises(ValueError):
        gqa.pages_resize_(t, t[:, 0].contiguous(), t[:, 0].contiguous(), 16)
    with pytest.raises(ValueError):
        gqa.cache8(4, 2, 64, page=16, block=48)
