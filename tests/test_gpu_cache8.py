"""The paged 8-bit K/V cache on the GPU against the double oracle: quantised
bytes, scales, page tables and moved pages bit for bit, decode within the bound
that oracle.cache8.decode derives for its arithmetic."""

import threading

import numpy as np
import pytest
import torch

import grouped_query_attention_attn_b200 as gqa
from grouped_query_attention_attn_b200 import _binding
from oracle import cache8 as oc
from oracle import ref

pytestmark = pytest.mark.gpu

KINDS = ["e4m3", "int8"]
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def to_gpu(p):
    t = [torch.from_numpy(p[n].copy()).cuda().view(DTYPE[p["kind"]]) for n in ("k", "v")]
    return gqa.Cache8(*t, *(torch.from_numpy(p[n].copy()).cuda() for n in ("k_scale", "v_scale")))


def same(cache, p):
    for n in ("k", "v"):
        got = getattr(cache, n).view(torch.uint8).cpu().numpy()
        assert np.array_equal(got, p[n]), (n, np.argwhere(got != p[n])[:3], int((got != p[n]).sum()))
    for n in ("k_scale", "v_scale"):
        assert np.array_equal(getattr(cache, n).cpu().numpy(), p[n]), n


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(rng, shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)


def random_table(rng, B, M, n_pages, held):
    ids = rng.permutation(n_pages)[:B * M].reshape(B, M)
    return [[int(ids[b, s]) if s < held[b] else -1 for s in range(M)] for b in range(B)]


def make(seed, kind, Hkv, d, page, block, lens, M=None, extra=0, spread=1.0):
    """A filled pool, a shuffled table for lens (+ extra rows each) and the rng."""
    rng = np.random.default_rng(seed)
    M = M or max(1, max(-(-(n + extra) // page) for n in lens))
    n_pages = len(lens) * M + 2
    p = oc.pool(n_pages, Hkv, page, d, block, kind, rng, spread)
    table = random_table(rng, len(lens), M, n_pages, [-(-(n + extra) // page) for n in lens])
    return rng, p, table


def spoil(p, table, lens):
    """NaN / largest bytes in every row and NaN scales in every block that no sequence's row needs."""
    used = np.zeros(p["k"].shape[:1] + p["k"].shape[2:3], bool)
    for row, n in zip(table, lens):
        for j in range(n):
            used[row[j // p["page"]], j % p["page"]] = True
    blocks = used.reshape(used.shape[0], -1, p["block"]).any(-1)
    for n in ("k", "v"):
        p[n][np.broadcast_to(~used[:, None], p[n].shape[:3])] = 127
        p[n + "_scale"][np.broadcast_to(~blocks[:, None], p[n + "_scale"].shape)] = np.nan


def check_decode(p, table, lens, q, scale=None, window=None, sinks=0, **kw):
    d = q.shape[-1]
    o = gqa.decode8(q.cuda(), to_gpu(p), ints(table), ints(lens), scale=scale, window=window, sinks=sinks, **kw)
    gqa.device_status()
    want, bound = oc.decode(p, table, lens, q.double().numpy(), scale or d ** -0.5, window or 0, sinks)
    got = o.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - want) / bound)
    assert worst <= 1.0, worst
    return o


# ------------------------------------------------------------------ decode --

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (8, 2, 64), (3, 3, 128), (7, 1, 64), (16, 1, 128),
                                      (17, 1, 128), (32, 1, 64), (32, 1, 128), (64, 2, 64)])
def test_decode_heads(gqa_lib, kind, Hq, Hkv, d):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 130, 700]
    rng, p, table = make(Hq + d, kind, Hkv, d, 64, 32, lens)
    spoil(p, table, lens)
    o = check_decode(p, table, lens, bf16(rng, (len(lens), Hq, d)))
    assert torch.all(o[1] == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (32, 32), (48, 16), (48, 48), (80, 80), (96, 32),
                                        (128, 64), (256, 256), (1024, 16), (192, 192)])
def test_decode_pages(gqa_lib, page, block, d):
    lens = [5, page, page + 1, 2 * page - 1, 333]
    rng, p, table = make(page + block, "e4m3", 2, d, page, block, lens, M=-(-400 // page) + 1)
    lens[3] = min(lens[3], (-(-400 // page) + 1) * page)
    spoil(p, table, lens)
    check_decode(p, table, lens, bf16(rng, (5, 6, d)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 0), (100, 64), (100, 65), (300, 200),
                                          (5, 1000), (100000, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_window(gqa_lib, window, sinks, d):
    lens = [1, 5, 64, 100, 101, 163, 299, 640, 0, 1333]
    rng, p, table = make(window % 1000 + sinks % 1000, "int8", 2, d, 32, 16, lens)
    spoil(p, table, lens)
    # pages without a visible row need not exist
    gone = [[e if any((j >= n - window) or j < sinks for j in range(s * 32, min(n, s * 32 + 32))) else -1
             for s, e in enumerate(row)] for row, n in zip(table, lens)]
    check_decode(p, gone, lens, bf16(rng, (len(lens), 8, d)), window=window, sinks=sinks)


def test_decode_many_splits(gqa_lib):
    # one sequence over the whole grid, and several of very different lengths
    for lens, M in (([40000], 700), ([20000, 1, 300], 320), ([1] * 130 + [3000], 50)):
        rng, p, table = make(len(lens), "e4m3", 1, 64, 64, 64, lens, M=M)
        check_decode(p, table, lens, bf16(rng, (len(lens), 3, 64)))


@pytest.mark.parametrize("kind", KINDS)
def test_decode_unequal_scales(gqa_lib, kind):
    # V scales that rise and fall by up to 2^40 from block to block, blocks of
    # scale 0, and queries far from 1
    lens = [64, 500, 1200]
    rng, p, table = make(5, kind, 2, 128, 32, 16, lens)
    p["k_scale"] *= 2.0 ** -3
    p["v_scale"] *= np.exp2(rng.integers(-20, 20, p["v_scale"].shape)).astype(np.float32)
    p["v_scale"][::3, :, 1] = 0.0
    q = bf16(rng, (3, 8, 128))
    for f, scale in ((1.0, None), (2.0 ** 100, 2.0 ** -104), (2.0 ** -100, 2.0 ** 97), (1.0, 3.0)):
        check_decode(p, table, lens, q * f, scale=scale)
    p["v_scale"][:] = 0.0
    assert torch.all(check_decode(p, table, lens, q) == 0)


def test_decode_scales_that_are_no_powers_of_two(gqa_lib):
    lens = [300, 77]
    rng, p, table = make(6, "int8", 2, 64, 64, 16, lens)
    p["k_scale"] *= rng.uniform(0.5, 1.5, p["k_scale"].shape).astype(np.float32)
    p["v_scale"] *= rng.uniform(0.1, 9.0, p["v_scale"].shape).astype(np.float32)
    check_decode(p, table, lens, bf16(rng, (2, 4, 64)))


def test_decode_nan_in_a_visible_row_reaches_its_group_only(gqa_lib):
    rng, p, table = make(7, "e4m3", 2, 128, 64, 64, [200, 200])
    p["v"][table[0][1], 1, 3, 5] = 127
    o = gqa.decode8(bf16(rng, (2, 8, 128)).cuda(), to_gpu(p), ints(table), ints([200, 200]))
    nan = torch.isnan(o)
    assert torch.all(nan[0, 4:, 5]) and int(nan.sum()) == 4


@pytest.mark.parametrize("d,Hq", [(128, 8), (64, 8), (128, 40)])
def test_decode_rope_is_rotation_then_decode(gqa_lib, d, Hq):
    lens = [1, 0, 100, 5000]
    rng, p, table = make(8, "e4m3", 2, d, 64, 64, lens)
    q, c, t, n = bf16(rng, (4, Hq, d)).cuda(), to_gpu(p), ints(table), ints(lens)
    got = gqa.decode8(q, c, t, n, rope_theta=10000.0, window=700, sinks=2)
    want = gqa.decode8(gqa.rope_decode_q_(q.clone(), n), c, t, n, window=700, sinks=2)
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_matches_bf16_decode_on_the_values(gqa_lib, kind):
    lens = [700, 64, 1, 333]
    rng, p, table = make(9, kind, 2, 128, 64, 16, lens)
    q, c, t, n = bf16(rng, (4, 8, 128)).cuda(), to_gpu(p), ints(table), ints(lens)
    k, v = gqa.cache8_read(c, t, n, 704)
    a, o = gqa.decode8(q, c, t, n), gqa.decode(q, k, v, n)
    # bf16 decode rounds its weights to 2^-8, twice in the quotient, and the output to 2^-8
    assert torch.all((a - o).abs() <= 2.0 ** -6 * v.abs().amax())


def test_decode_bad_entries_are_flagged_and_left_out(gqa_lib):
    lens = [300, 300]
    rng, p, table = make(10, "e4m3", 2, 128, 64, 64, lens)
    q = bf16(rng, (2, 8, 128))
    for e in (-1, len(p["k"]), 2 ** 31 - 1, -2 ** 31):
        t = [list(r) for r in table]
        t[0][2] = e
        o = gqa.decode8(q.cuda(), to_gpu(p), ints(t), ints(lens))
        assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
        want, bound = oc.decode(p, t, lens, q.double().numpy(), 128 ** -0.5)
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
    t = [[-1] * len(r) for r in table]
    assert torch.all(gqa.decode8(q.cuda(), to_gpu(p), ints(t), ints(lens)) == 0)
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    # lengths outside the table
    M = len(table[0]) * 64
    full = [list(rng.permutation(len(p["k"]))[:len(r)]) for r in table]
    o = gqa.decode8(q.cuda(), to_gpu(p), ints(full), ints([M + 1, -5]))
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    want, bound = oc.decode(p, full, [M, 0], q.double().numpy(), 128 ** -0.5)
    assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)


def test_decode_repeats_and_reuses_a_dirty_workspace(gqa_lib):
    lens = [3000, 100, 0, 1500]
    rng, p, table = make(11, "e4m3", 2, 128, 64, 64, lens)
    q, c, t, n = bf16(rng, (4, 8, 128)).cuda(), to_gpu(p), ints(table), ints(lens)
    want = gqa.decode8(q, c, t, n)
    need = gqa.decode8_workspace_size(4, 8, 2, 128, t.shape[1] * 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(gqa.decode8(q, c, t, n, workspace=ws), want)
    with pytest.raises(ValueError):
        gqa.decode8(q, c, t, n, workspace=ws[:need - 256])
    with pytest.raises(ValueError):
        gqa.decode8(q, c, t, n, workspace=ws[1:])


@pytest.mark.parametrize("Hq,Hkv,d", [(17, 1, 64), (31, 1, 128), (64, 2, 128), (12, 1, 128), (3, 3, 64)])
def test_decode_stays_in_its_workspace(gqa_lib, Hq, Hkv, d):
    # units in many pieces, groups shared by two CTAs; bytes past the workspace stay
    for lens in ([9000, 3, 0, 700], [1], [33] * 300):
        rng, p, table = make(13, "int8", Hkv, d, 48, 48, lens)
        q = bf16(rng, (len(lens), Hq, d))
        need = gqa.decode8_workspace_size(len(lens), Hq, Hkv, d, len(table[0]) * 48)
        ws = torch.full((need + 512,), 171, dtype=torch.uint8, device="cuda")
        o = check_decode(p, table, lens, q, workspace=ws[:need])
        assert torch.equal(check_decode(p, table, lens, q, rope_theta=None, workspace=ws[:need]), o)
        assert torch.all(ws[need:] == 171)


def test_decode_graphs_that_share_a_workspace(gqa_lib):
    lens = [3000, 100, 0, 1500]
    rng, p, table = make(12, "int8", 2, 128, 64, 64, lens)
    c, t = to_gpu(p), ints(table)
    n, q = ints(lens), bf16(rng, (4, 8, 128)).cuda()
    ws = torch.empty(gqa.decode8_workspace_size(4, 8, 2, 128, t.shape[1] * 64), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    gqa.decode8(q, c, t, n, workspace=ws)
    for i, o in enumerate(outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gqa.decode8(q, c, t, n, workspace=ws, out=o, window=500 if i else None)
        graphs.append(g)
    for cut in ([0, 0, 0, 0], [100, 5, 0, 700], [2999, 99, 0, 1]):
        n.copy_(ints([a - b for a, b in zip(lens, cut)]))
        q.copy_(bf16(rng, (4, 8, 128)))
        for g in graphs:
            g.replay()
        assert torch.equal(outs[0], gqa.decode8(q, c, t, n))
        assert torch.equal(outs[1], gqa.decode8(q, c, t, n, window=500))
    gqa.device_status()


def test_decode_from_two_threads_on_two_streams(gqa_lib):
    lens = [2000, 100, 900]
    rng, p, table = make(13, "e4m3", 4, 128, 64, 16, lens)
    c, t, n = to_gpu(p), ints(table), ints(lens)
    qs = [bf16(rng, (3, 16, 128)).cuda() for _ in range(2)]
    want = [gqa.decode8(q, c, t, n) for q in qs]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = gqa.decode8(qs[i], c, t, n)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ append --

def check_append(p, table, lens, counts, k, v, given=True):
    c = to_gpu(p)
    gqa.cache8_append_(c, ints(table), ints(lens), k.cuda(), v.cuda(), counts=ints(counts) if given else None)
    gqa.device_status()
    oc.append(p, table, lens, counts, k.double().numpy(), v.double().numpy())
    same(c, p)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (48, 48), (64, 16), (64, 32), (64, 64), (128, 128), (256, 256),
                                        (96, 48), (80, 80), (112, 112)])
def test_append_ragged(gqa_lib, kind, d, page, block):
    T = 70
    lens, counts = [0, 5, 16, 63, 130, 7, 200], [70, 1, 0, 33, 17, 64, 70]
    rng, p, table = make(page + block + d, kind, 3, d, page, block, lens, extra=T)
    k, v = bf16(rng, (7, T, 3, d), 3.0), bf16(rng, (7, T, 3, d), 0.01)
    check_append(p, table, lens, counts, k, v)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("std", [1e-3, 1.0, 1e3])
def test_append_single_tokens(gqa_lib, kind, std):
    # one row to each sequence at every offset of a block: the scale grows or stays
    lens = list(range(0, 67))
    rng, p, table = make(17, kind, 2, 128, 32, 32, lens, extra=1)
    k, v = bf16(rng, (67, 1, 2, 128), std), bf16(rng, (67, 1, 2, 128), std)
    check_append(p, table, lens, [1] * 67, k, v, given=False)


@pytest.mark.parametrize("kind", KINDS)
def test_append_token_by_token_keeps_every_row_close(gqa_lib, kind):
    rng = np.random.default_rng(18)
    p = oc.pool(4, 2, 32, 64, 16, kind)
    c, table = to_gpu(p), [[2, 0, 3]]
    x = bf16(rng, (1, 90, 2, 64)) * torch.exp2(torch.randint(-6, 6, (1, 90, 1, 1)).float())
    x = x.to(torch.bfloat16)
    for i in range(90):
        row = x[:, i:i + 1].contiguous()
        gqa.cache8_append_(c, ints(table), ints([i]), row.cuda(), (-row).cuda())
        oc.append(p, table, [i], [1], row.double().numpy(), -row.double().numpy())
    same(c, p)


@pytest.mark.parametrize("kind", KINDS)
def test_append_special_values(gqa_lib, kind):
    rng, p, table = make(19, kind, 2, 128, 64, 16, [3, 16], extra=64)
    k, v = bf16(rng, (2, 64, 2, 128)), bf16(rng, (2, 64, 2, 128))
    k[0, 2, 0, 7], k[0, 3, 1, 9], k[1, 1, 0, 3] = float("inf"), float("-inf"), float("nan")
    v[0] = 0.0                                            # blocks of zeros
    v[1, :16, 0] = float("inf")                           # nothing finite in the block
    v[1, 16:32] = 2.0 ** -130                             # subnormal
    v[1, 32:48] = 3.38e38                                 # the largest
    v[1, 48:64, :, 1:] = 0.0
    v[1, 48:64, :, 0] = float("-inf")
    check_append(p, table, [3, 16], [64, 64], k, v)


def test_append_a_scale_that_is_no_power_of_two(gqa_lib):
    rng, p, table = make(20, "int8", 1, 64, 32, 32, [10, 20], extra=5)
    p["k_scale"] *= np.float32(1.25)
    k, v = bf16(rng, (2, 5, 1, 64), 0.01), bf16(rng, (2, 5, 1, 64), 100.0)
    c = to_gpu(p)
    gqa.cache8_append_(c, ints(table), ints([10, 20]), k.cuda(), v.cuda())
    # the larger old scale stays, and its rows with it
    for b, n in ((0, 10), (1, 20)):
        assert torch.equal(c.k_scale[table[b][0]].cpu(), torch.from_numpy(p["k_scale"][table[b][0]]))
        assert np.array_equal(c.k[table[b][0], :, :n].view(torch.uint8).cpu().numpy(), p["k"][table[b][0], :, :n])


def test_append_leaves_other_rows_and_flags_bad_ones(gqa_lib):
    lens = [30, 60, 10, 5, 5]
    rng, p, table = make(21, "e4m3", 2, 128, 32, 16, lens, extra=10)
    k, v = bf16(rng, (5, 10, 2, 128)), bf16(rng, (5, 10, 2, 128))
    bad = [list(r) for r in table]
    bad[0][1] = -1                                        # rows 32 .. 39 have no page
    bad[1][1] = len(p["k"])                               # rows 60 .. 63 neither
    c = to_gpu(p)
    gqa.cache8_append_(c, ints(bad), ints([30, 60, 10, -1, 5]), k.cuda(), v.cuda(), counts=ints([10, 10, 10, 10, 11]))
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    kd, vd = k.double().numpy(), v.double().numpy()
    oc.append(p, [table[0]], [30], [2], kd[:1], vd[:1])
    oc.append(p, [table[1]], [64], [6], kd[1:2, 4:], vd[1:2, 4:])
    oc.append(p, [table[2]], [10], [10], kd[2:3], vd[2:3])
    same(c, p)
    # rows past the table's slots
    M = len(table[0]) * 32
    gqa.cache8_append_(c, ints(table), ints([M] * 5), k.cuda(), v.cuda())
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    same(c, p)


# -------------------------------------------------------------- read, copy --

def test_append_of_no_rows_needs_no_page(gqa_lib):
    # rows that add nothing, ending inside a block: their pages may be gone or be shared
    rng, p, table = make(16, "e4m3", 2, 128, 64, 16, [5, 70, 23], extra=20)
    c, lens, counts = to_gpu(p), [5, 70, 23], [0, 0, 9]
    k, v = bf16(rng, (3, 9, 2, 128)), bf16(rng, (3, 9, 2, 128))
    gone = [[-1] * len(table[0]), [table[1][0], table[2][0]] + [-1] * (len(table[1]) - 2), table[2]]
    gqa.cache8_append_(c, ints(gone), ints(lens), k.cuda(), v.cuda(), ints(counts))
    gqa.device_status()
    oc.append(p, [table[2]], [23], [9], k[2:].double().numpy(), v[2:].double().numpy())
    same(c, p)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block,T", [(16, 16, 1), (48, 16, 100), (64, 32, 333), (128, 128, 17), (1024, 256, 40)])
def test_read(gqa_lib, kind, d, page, block, T):
    lens = [0, 1, 16, 100, 333]
    rng, p, table = make(T + d, kind, 3, d, page, block, lens)
    spoil(p, table, lens)
    out = [torch.full((5, T, 3, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = gqa.cache8_read(to_gpu(p), ints(table), ints(lens), T, out=out)
    gqa.device_status()
    for name, x in (("k", k), ("v", v)):
        for b, n in enumerate(lens):
            n = min(n, T)
            want = torch.from_numpy(oc.rows(p, name, table, b, n)).to(torch.bfloat16)
            assert torch.equal(x[b, :n].cpu(), want) and torch.all(x[b, n:] == 0)


def test_read_flags_bad_entries(gqa_lib):
    rng, p, table = make(30, "int8", 2, 64, 16, 16, [40, 40])
    table[0][1] = -1
    k, _ = gqa.cache8_read(to_gpu(p), ints(table), ints([40, 1000]), 40)
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    assert torch.all(k[0, 16:32] == 0) and torch.all(k[0, 32:40].abs().sum(-1) > 0)


@pytest.mark.parametrize("page,block,d", [(16, 16, 64), (48, 16, 128), (64, 64, 128), (1024, 256, 64)])
def test_copy(gqa_lib, page, block, d):
    rng = np.random.default_rng(page)
    p = oc.pool(9, 3, page, d, block, "e4m3", rng)
    moves = [(0, 8, page), (0, 7, 1), (2, 3, page - 1), (5, 1, 0)]
    c = to_gpu(p)
    gqa.cache8_copy_(c, ints([[4, 0, 0], *moves, [1, 2, 3], [-7, 100, 1000]]))
    gqa.device_status()
    oc.copy(p, moves)
    same(c, p)
    gqa.cache8_copy_(c, ints([[0, 0, 0]]))
    gqa.cache8_copy_(c, ints([[4, 0, 0], (0, 9, 1), (-1, 1, 1), (1, 2, page + 1), (6, 4, 2)]))
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    oc.copy(p, [(6, 4, 2)])
    same(c, p)
    gqa.cache8_copy_(c, ints([[3, 0, 0], (3, 5, 2)]))
    assert _binding.gqa_device_status(1) != 0
    gqa.cache8_copy_(c, ints([[-3, 0, 0], (3, 6, 2)]))
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    oc.copy(p, [(3, 5, 2)])
    same(c, p)


# ------------------------------------------------------------------- pages --

def lists(t):
    return t.cpu().tolist()


def moves_of(m):
    m = m.cpu().tolist()
    assert m[0][1:] == [0, 0]
    return [tuple(x) for x in m[1:1 + m[0][0]]]


@pytest.mark.parametrize("B,M,n_pages,page", [(1, 1, 1, 16), (3, 4, 13, 16), (8, 40, 200, 48), (5, 3, 100, 1),
                                              (300, 33, 9000, 64), (1, 20000, 30000, 64), (2000, 1, 1500, 16)])
def test_pages_sequence(gqa_lib, B, M, n_pages, page):
    # resize, fork, compact in turn, each against the lists; the pool may run out
    rng = np.random.default_rng(B + M)
    table, refs = [[-1] * M for _ in range(B)], [0] * n_pages
    t, r = ints(table), ints(refs)
    for step in range(6):
        room = n_pages * page / B * (0.5 if step % 2 else 0.9)
        lens = [int(min(M * page, x)) for x in rng.exponential(room, B)]
        missing = oc.resize(table, refs, lens, page)
        gqa.pages_resize_(t, r, ints(lens), page)
        assert _binding.gqa_device_status(1) == (_binding.GQA_ERR_PAGES if missing else 0)
        assert lists(t) == table and lists(r) == refs
        # a sequence ends where its pages do
        lens = [min(n, page * next((s for s, e in enumerate(x) if e < 0), M)) for n, x in zip(lens, table)]
        parents = [int(x) for x in rng.integers(-1, B, B)]
        for b in rng.permutation(B)[:B // 3]:
            parents[b] = int(b)
        n = ints(lens)
        oc.resize(table, refs, lens, page)
        gqa.pages_resize_(t, r, n, page)
        wants = sum(x >= 0 for x in parents)
        got = moves_of(gqa.pages_fork_(t, r, n, ints(parents), page))
        want = oc.fork(table, refs, lens, parents, page)
        assert _binding.gqa_device_status(1) in (0, _binding.GQA_ERR_PAGES)
        assert got == want and len(got) <= wants
        assert lists(t) == table and lists(r) == refs and lists(n) == lens
        got = moves_of(gqa.pages_compact_(t, r, page))
        assert got == oc.compact(table, refs, page)
        gqa.device_status()
        assert lists(t) == table and lists(r) == refs


def test_pages_resize_edges(gqa_lib):
    t, r = ints([[0, -1, 2, 3], [2, 1, -1, -1]]), ints([1, 1, 2, 1, 0, 0])
    gqa.pages_resize_(t, r, ints([64, 16]), 16)          # a hole is filled, a shared page dropped once
    gqa.device_status()
    assert lists(t) == [[0, 1, 2, 3], [2, -1, -1, -1]] and lists(r) == [1, 1, 2, 1, 0, 0]
    gqa.pages_resize_(t, r, ints([65, -1]), 16)          # lengths outside the table are clamped
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    assert lists(t) == [[0, 1, 2, 3], [-1] * 4] and lists(r) == [1, 1, 1, 1, 0, 0]
    t[1, 0], t[1, 3] = 6, 2 ** 31 - 1                     # entries beyond the pool count as none
    gqa.pages_resize_(t, r, ints([64, 16]), 16)
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    assert lists(t) == [[0, 1, 2, 3], [4, -1, -1, -1]] and lists(r) == [1, 1, 1, 1, 1, 0]
    t[1, 1] = 5                                           # released without a reference
    gqa.pages_resize_(t, r, ints([64, 16]), 16)
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    empty = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    gqa.pages_resize_(empty, r, ints([]), 16)
    assert moves_of(gqa.pages_fork_(empty, r, ints([]), ints([]), 16)) == []
    with pytest.raises(ValueError):
        gqa.pages_resize_(t, r, ints([1]), 16)
    with pytest.raises(ValueError):
        gqa.pages_resize_(t, r, ints([1, 1]), 0)


def test_pages_fork_edges(gqa_lib):
    # row 0 has pages past its length: they stay with the row that goes on in them
    t, r, n = ints([[0, 1, 2, 3], [4, -1, -1, -1], [5, -1, -1, -1]]), ints([1] * 6 + [0] * 4), ints([20, 16, 3])
    m = gqa.pages_fork_(t, r, n, ints([2, 0, 0]), 16)
    gqa.device_status()
    # row 0 <- row 2 (its first child), row 1 <- row 0 (heir), row 2 <- row 0: a page for 4 rows
    assert moves_of(m) == [(1, 4, 4)]
    assert lists(t) == [[5, -1, -1, -1], [0, 1, 2, 3], [0, 4, -1, -1]]
    assert lists(r) == [2, 1, 1, 1, 1, 1, 0, 0, 0, 0] and lists(n) == [3, 20, 20]
    m = gqa.pages_fork_(t, r, n, ints([7, -9, 1]), 16)    # a parent that is no row, and none
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    assert moves_of(m) == [] and lists(n) == [0, 0, 20]
    assert lists(t) == [[-1] * 4, [-1] * 4, [0, 1, 2, 3]] and lists(r) == [1, 1, 1, 1] + [0] * 6


def test_pages_compact_flags_an_entry_without_a_reference(gqa_lib):
    t, r = ints([[3, 5], [9, -1]]), ints([0, 0, 0, 1, 0, 0])
    assert moves_of(gqa.pages_compact_(t, r, 16)) == [(3, 0, 16)]
    assert _binding.gqa_device_status(1) == _binding.GQA_ERR_INVALID_ARG
    assert lists(t) == [[0, 5], [9, -1]] and lists(r) == [1, 0, 0, 0, 0, 0]


# ------------------------------------------------------ together, and graphs --

@pytest.mark.parametrize("kind,d,page,block", [("e4m3", 128, 64, 32), ("int8", 64, 16, 16), ("e4m3", 64, 48, 48)])
def test_a_run_of_them(gqa_lib, kind, d, page, block):
    """Prompts in, then decode steps with forks, sequences that leave and enter, and
    compactions, over two layers that share the table; all against the oracle."""
    rng = np.random.default_rng(d + page)
    B, Hkv, Hq, M, n_pages = 5, 2, 6, 5, 19
    layers = [oc.pool(n_pages, Hkv, page, d, block, kind) for _ in range(2)]
    caches = [gqa.cache8(n_pages, Hkv, d, page, block, DTYPE[kind]) for _ in range(2)]
    table, refs, lens = [[-1] * M for _ in range(B)], [0] * n_pages, [0] * B
    t, r, n = ints(table), ints(refs), ints(lens)

    def move(m, want):
        assert moves_of(m) == want
        for c, p in zip(caches, layers):
            gqa.cache8_copy_(c, m)
            oc.copy(p, want)

    def add(counts):
        T = max(counts)
        to = [a + b for a, b in zip(lens, counts)]
        assert oc.resize(table, refs, to, page) == 0
        gqa.pages_resize_(t, r, ints(to), page)
        for c, p in zip(caches, layers):
            k, v = bf16(rng, (B, T, Hkv, d), 2.0), bf16(rng, (B, T, Hkv, d))
            gqa.cache8_append_(c, t, n, k.cuda(), v.cuda(), counts=ints(counts))
            oc.append(p, table, lens, counts, k.double().numpy(), v.double().numpy())
        lens[:] = to
        n.add_(ints(counts))

    add([page + 3, 10, 2 * page, 0, 1])
    for step in range(6):
        add([1 if x else 0 for x in lens])
        if step == 1:
            parents = [0, 0, 2, 1, 2]
            move(gqa.pages_fork_(t, r, n, ints(parents), page), oc.fork(table, refs, lens, parents, page))
        if step == 3:
            lens[0] = lens[2] = 0
            n.copy_(ints(lens))
            oc.resize(table, refs, lens, page)
            gqa.pages_resize_(t, r, n, page)
            move(gqa.pages_compact_(t, r, page), oc.compact(table, refs, page))
            add([7, 0, page, 0, 0])
        assert lists(t) == table and lists(r) == refs and lists(n) == lens
        for c, p in zip(caches, layers):
            q = bf16(rng, (B, Hq, d))
            o = gqa.decode8(q.cuda(), c, t, n, window=40 if step % 2 else None, sinks=2)
            want, bound = oc.decode(p, table, lens, q.double().numpy(), d ** -0.5, 40 if step % 2 else 0, 2)
            assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
    gqa.device_status()


def test_prompt_chunks_through_the_cache(gqa_lib):
    # a prompt in two chunks: the second attends to the first's quantised rows
    # (cache8_read) and its own, as attn on the same values does
    rng = np.random.default_rng(40)
    c, t = gqa.cache8(8, 2, 128), ints([[3, 1, 6, 0]])
    k, v, q = (bf16(rng, (1, 200, h, 128)).cuda() for h in (2, 2, 8))
    gqa.rope_qk_(q, k)
    gqa.cache8_append_(c, t, ints([0]), k[:, :130].contiguous(), v[:, :130].contiguous())
    gqa.cache8_append_(c, t, ints([130]), k[:, 130:].contiguous(), v[:, 130:].contiguous())
    kk, vv = gqa.cache8_read(c, t, ints([200]), 200)
    o = gqa.attn(q[:, 130:].contiguous(), kk, vv)
    want, _ = ref.attn_fwd(q[:, 130:].cpu(), kk.cpu(), vv.cpu(), causal=True)
    assert np.max(np.abs(o.float().cpu().numpy() - want)) <= 2e-2
    # the last row is what decode8 gives for it
    o8 = gqa.decode8(q[:, 199].contiguous(), c, t, ints([200]))
    assert np.max(np.abs(o8.float().cpu().numpy() - want[:, -1])) <= 2e-2


def test_a_captured_step(gqa_lib):
    # fork, copy, resize, append and decode captured once and replayed on new data
    rng = np.random.default_rng(41)
    B, Hkv, Hq, d, page, n_pages, M = 4, 2, 8, 128, 16, 40, 8
    p = oc.pool(n_pages, Hkv, page, d, 16, "e4m3", rng)
    table, refs, lens = [[-1] * M for _ in range(B)], [0] * n_pages, [20, 33, 16, 5]
    oc.resize(table, refs, lens, page)
    c, t, r, n = to_gpu(p), ints(table), ints(refs), ints(lens)
    parents, n1 = ints([0, 1, 2, 3]), torch.empty(B, dtype=torch.int32, device="cuda")
    k, v, q = (torch.empty(s, dtype=torch.bfloat16, device="cuda")
               for s in ((B, 1, Hkv, d), (B, 1, Hkv, d), (B, Hq, d)))
    o = torch.empty_like(q)

    def step():
        gqa.cache8_copy_(c, gqa.pages_fork_(t, r, n, parents, page))
        torch.add(n, 1, out=n1)
        gqa.pages_resize_(t, r, n1, page)
        gqa.cache8_append_(c, t, n, k, v)
        gqa.decode8(q, c, t, n1, out=o)
        n.copy_(n1)

    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    gqa.device_status()
    with torch.cuda.stream(side):
        for i in range(8):
            if i == 1:
                with torch.cuda.graph(g, stream=side):
                    step()
            x = [bf16(rng, s.shape) for s in (k, v, q)]
            for a, b in zip((k, v, q), x):
                a.copy_(b)
            par = [int(y) for y in rng.integers(0, B, B)]
            parents.copy_(torch.tensor(par, dtype=torch.int32))
            g.replay() if i else step()
            oc.copy(p, oc.fork(table, refs, lens, par, page))
            oc.resize(table, refs, [y + 1 for y in lens], page)
            oc.append(p, table, lens, [1] * B, x[0].double().numpy(), x[1].double().numpy())
            lens = [y + 1 for y in lens]
            want, bound = oc.decode(p, table, lens, x[2].double().numpy(), d ** -0.5)
            assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
            assert lists(t) == table and lists(r) == refs and lists(n) == lens
    same(c, p)
    gqa.device_status()


def test_a_capture_over_two_streams(gqa_lib):
    # K / V appended on one stream, the table kept on another, joined before the decode
    rng = np.random.default_rng(42)
    p = oc.pool(20, 2, 64, 128, 64, "int8", rng)
    table, refs, lens = [[-1] * 4 for _ in range(3)], [0] * 20, [64, 100, 30]
    oc.resize(table, refs, [n + 1 for n in lens], 64)
    c, t, r, n = to_gpu(p), ints([[-1] * 4 for _ in range(3)]), ints([0] * 20), ints(lens)
    n1 = n + 1
    k, v, q = bf16(rng, (3, 1, 2, 128)), bf16(rng, (3, 1, 2, 128)), bf16(rng, (3, 8, 128))
    oc.append(p, table, lens, [1] * 3, k.double().numpy(), v.double().numpy())
    want, bound = oc.decode(p, table, [x + 1 for x in lens], q.double().numpy(), 128 ** -0.5)
    k, v, q = k.cuda(), v.cuda(), q.cuda()
    o = torch.empty_like(q)
    other = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        gqa.pages_resize_(t, r, n1, 64)
        other.wait_stream(here)
        with torch.cuda.stream(other):
            gqa.cache8_append_(c, t, n, k, v)
        gqa.pages_resize_(t, r, n1, 64)                   # nothing to do
        here.wait_stream(other)
        gqa.decode8(q, c, t, n1, out=o)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        o.zero_()
        g.replay()
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
    assert lists(t) == table and lists(r) == refs
    same(c, p)
    gqa.device_status()


def test_sequences_that_share_their_pages(gqa_lib):
    rng, p, table = make(43, "e4m3", 2, 128, 64, 64, [500, 300])
    t, n = ints([table[0], table[1], table[0], table[0]]), ints([500, 300, 499, 64])
    q = bf16(rng, (4, 8, 128))
    o = gqa.decode8(q.cuda(), to_gpu(p), t, n)
    want, bound = oc.decode(p, lists(t), lists(n), q.double().numpy(), 128 ** -0.5)
    assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)


def test_many_sequences(gqa_lib):
    # the most that one append takes, one row each: the weight of a lone row is 1
    B = 65535
    c = gqa.cache8(B, 1, 64, page=16, block=16, dtype=torch.int8)
    t = torch.randperm(B, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).int().view(B, 1)
    refs = torch.zeros(B, dtype=torch.int32, device="cuda")
    v = torch.randint(-127, 128, (B, 1, 1, 64), device="cuda").to(torch.bfloat16)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    gqa.cache8_append_(c, t, zero, v, v)
    k2, v2 = gqa.cache8_read(c, t, zero + 1, 1)
    assert torch.equal(k2, v) and torch.equal(v2, v)
    o = gqa.decode8(v[:, 0].expand(B, 4, 64).contiguous(), c, t, zero + 1)
    assert torch.equal(o, v[:, 0].expand(B, 4, 64))
    t.fill_(-1)
    gqa.pages_resize_(t, refs, zero + 16, 16)
    assert torch.equal(t[:, 0], torch.arange(B, device="cuda").int()) and torch.all(refs == 1)
    gqa.device_status()


def test_large_offsets(gqa_lib):
    # pages past 2^32 bytes of the pool: 36000 pages of 128 KB
    need = 36000 * 8 * 128 * 128 * 2
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("not enough free device memory")
    rng = np.random.default_rng(50)
    c = gqa.cache8(36000, 8, 128, page=128, block=128)
    small = oc.pool(4, 8, 128, 128, 128, "e4m3")
    ids, lens = [35999, 20000, 34001, 1], [0]
    table = [ids[:3]]
    k, v = bf16(rng, (1, 300, 8, 128)), bf16(rng, (1, 300, 8, 128))
    gqa.cache8_append_(c, ints(table), ints(lens), k.cuda(), v.cuda())
    oc.append(small, [[0, 1, 2]], [0], [300], k.double().numpy(), v.double().numpy())
    gqa.cache8_copy_(c, ints([[1, 0, 0], [34001, 1, 44]]))
    for at, e in ((0, 35999), (1, 20000), (2, 34001)):
        assert np.array_equal(c.k[e].view(torch.uint8).cpu().numpy(), small["k"][at])
    assert np.array_equal(c.v[1, :, :44].view(torch.uint8).cpu().numpy(), small["v"][2, :, :44])
    q = bf16(rng, (1, 32, 128))
    o = gqa.decode8(q.cuda(), c, ints(table), ints([300]))
    want, bound = oc.decode(small, [[0, 1, 2]], [300], q.double().numpy(), 128 ** -0.5)
    assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
    x, _ = gqa.cache8_read(c, ints(table), ints([300]), 300)
    assert torch.equal(x[0].cpu(), torch.from_numpy(oc.rows(small, "k", [[0, 1, 2]], 0, 300)).to(torch.bfloat16))
    gqa.device_status()
