"""decode8 over the whole range of V scales that the cache may hold (0 or >= 2^-126), with
scales that fall far and more than once within the keys of one warp."""

import numpy as np
import pytest
import torch

import grouped_query_attention_attn_b200 as gqa
from oracle import cache8 as oc
from test_gpu_cache8 import KINDS, bf16, check_decode, ints, make, to_gpu
from test_oracle_cache8_bound import case as long_case

pytestmark = pytest.mark.gpu

# exponent of the V scale of a sequence's i-th block of 16 keys
PATTERNS = {
    "then_least": lambda i, n: 0 if i < n // 2 else -126,
    "one_block": lambda i, n: -126 if i // 2 == n // 4 else -5,
    "halves": lambda i, n: (0, -70)[i % 2],
    "steps": lambda i, n: (-7, -70, -126)[3 * i // n],
    "every_tile": lambda i, n: (-7, -71, -126, -7)[i // 2 % 4],
    "stairs": lambda i, n: 100 - 226 * i // n,
    "up_and_down": lambda i, n: (-126, 0, -126, 60, -40, -126)[6 * i // n],
    "zeros_between": lambda i, n: (-3, None, -126)[i % 3],
}


def set_scales(p, table, lens, pattern):
    for row, n in zip(table, lens):
        blocks = -(-n // p["block"])
        per = p["page"] // p["block"]
        for i in range(blocks):
            e = PATTERNS[pattern](i, blocks)
            p["v_scale"][row[i // per], :, i % per] = 0.0 if e is None else 2.0 ** e


def check_many(p, table, lens, q, want=None):
    """The sequences, 27 times over so that every warp takes several tiles of a unit."""
    n, d = 27, q.shape[-1]
    o = gqa.decode8(q.repeat(n, 1, 1).cuda(), to_gpu(p), ints(table * n), ints(lens * n))
    gqa.device_status()
    want, bound = want or oc.decode(p, table, lens, q.double().numpy(), d ** -0.5)
    off = np.abs(o.double().cpu().numpy().reshape(n, *want.shape) - want)
    assert np.all(off <= bound), np.nanmax(off / bound)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("G,d", [(2, 128), (9, 128), (2, 64), (9, 64)])
def test_v_scales_that_fall(gqa_lib, kind, pattern, G, d):
    lens = [700, 550, 401]
    rng, p, table = make(len(pattern) + d, kind, 4, d, 32, 16, lens)
    set_scales(p, table, lens, pattern)
    check_many(p, table, lens, bf16(rng, (3, 4 * G, d)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_all_the_weight_on_small_values(gqa_lib, kind, d):
    # the keys of the second half, with V 2^-60 times the first's, take all the weight:
    # the output is theirs, to its own precision
    lens = [512, 512, 384]
    rng, p, table = make(3, kind, 4, d, 32, 16, lens)
    for row, n in zip(table, lens):
        for i in range(n // 16):
            late = i >= n // 32
            p["v_scale"][row[i // 2], :, i % 2] = 2.0 ** (-60 if late else 0)
            p["k_scale"][row[i // 2], :, i % 2] = 2.0 ** (0 if late else -126)
    # keys of one sign, so that the late ones score 130 and more and the others 0: these
    # have weights below 2^-186, nothing even against values 2^-60 of theirs
    k = np.minimum(np.ceil(np.abs(oc.values(p["k"], kind))), 32.0) + 32.0
    p["k"][:] = oc.encode(k, kind)
    q = torch.full((3, 8, d), 0.5).to(torch.bfloat16)
    late = [row[n // 64:] for row, n in zip(table, lens)]
    check_many(p, table, lens, q, oc.decode(p, late, [n // 2 for n in lens], q.double().numpy(), d ** -0.5))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [20, 600, 9000])
def test_nan_stays_nan_in_one_piece_and_in_many(gqa_lib, d, n):
    # a query with a NaN, and keys of which every group has one: the rows they reach are
    # NaN, whether their sequence is read by one CTA or cut into pieces; the others stand
    rng, p, table = make(n + d, "e4m3", 2, d, 32, 16, [n, n])
    q = bf16(rng, (2, 8, d))
    q[0, 3, 5] = float("nan")
    want, bound = oc.decode(p, table, [n, n], q.nan_to_num(0.0).double().numpy(), d ** -0.5)
    for e in table[1]:
        p["k"][e, 1, ::7, 9] = 127
    o = gqa.decode8(q.cuda(), to_gpu(p), ints(table), ints([n, n])).double().cpu().numpy()
    gqa.device_status()
    nan = np.zeros(o.shape, bool)
    nan[0, 3] = nan[1, 4:] = True
    assert np.array_equal(np.isnan(o), nan)
    assert np.all(np.abs(o - want)[~nan] <= bound[~nan])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,d", [(2, 128), (9, 128), (2, 64), (9, 64)])
def test_small_weights_keep_their_precision(gqa_lib, kind, G, d):
    # of 32 keys one has weight 1 and V = 0, and 16 have weight 2^-14.7 and all of V, in a
    # block whose V scale is 64 times smaller.  Their weights are within half a step of
    # f16, 2^-11, and what their scores are off, 2^-20 of 14.7; then bf16's half step 2^-8
    n, turn = 640, 0.98046875                             # the query, in bf16; log2 units
    p = oc.pool(n // 32, 1, 32, d, 16, kind)
    p["k"][:, 0, :, 0] = oc.encode(-15.0, kind)
    p["k"][:, 0, 0, 0] = oc.encode(0.0, kind)
    p["v"][:, 0, 16:] = oc.encode(96.0, kind)
    p["k_scale"][:] = 1.0
    p["v_scale"][:] = [1.0, 2.0 ** -6]
    q = torch.zeros((40, G, d), dtype=torch.bfloat16)
    q[..., 0] = turn
    o = gqa.decode8(q.cuda(), to_gpu(p), ints([list(range(n // 32))] * 40), ints([n] * 40), scale=float(np.log(2.0)))
    gqa.device_status()
    w = 2.0 ** (-15 * turn)
    want = 16 * w * 96 * 2.0 ** -6 / (1 + 31 * w)
    assert np.max(np.abs(o.double().cpu().numpy() / want - 1)) <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,d", [(2, 128), (9, 128), (2, 64), (9, 64)])
def test_queries_at_the_small_end_of_bf16(gqa_lib, kind, G, d):
    # the largest element of a row is subnormal, or just normal; scale brings the scores to 1
    lens = [300, 33]
    rng, p, table = make(G + d, kind, 2, d, 32, 16, lens)
    for f, scale in ((2.0 ** -131, 2.0 ** 127), (2.0 ** -126, 2.0 ** 123)):
        q = (bf16(rng, (2, 2 * G, d)).float().clamp(-3, 3) * f).to(torch.bfloat16)
        assert int((q != 0).sum()) > q.numel() // 2
        check_decode(p, table, lens, q, scale=scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("few", [False, True])
def test_values_at_the_end_of_the_range(gqa_lib, kind, d, few):
    # V up to 1.75 x 2^127: any sum of two is past fp32, their means are not.  few: one block
    # in nine, the others 2^139 below
    lens = [1, 20, 700, 9000]
    rng, p, table = make(d + few, kind, 2, d, 32, 16, lens)
    for row, n in zip(table, lens):
        for i in range(-(-n // 16)):
            p["v_scale"][row[i // 2], :, i % 2] = 2.0 ** (-20 if few and i % 9 else 119)
    check_decode(p, table, lens, bf16(rng, (4, 6, d)))


@pytest.mark.parametrize("G", [1, 6, 20])
@pytest.mark.parametrize("n,d", [(9000, 128), (20000, 64), (40000, 64)])
def test_pieces_whose_values_differ(gqa_lib, n, d, G):
    # every page has V of its own: a page lost or read twice is at least twice the bound
    # (test_oracle_cache8_bound)
    p, pages, q = long_case(n, d, n + 1, True)
    rng = np.random.default_rng(G)
    q = np.concatenate([q] + [np.round(rng.standard_normal((1, 1, d)) * 64) / 64 for _ in range(G - 1)], 1)
    q = torch.from_numpy(q).to(torch.bfloat16)
    for lens in ([n], [n, 100, n - 7]):
        check_decode(p, [pages] * len(lens), lens, q.repeat(len(lens), 1, 1))
