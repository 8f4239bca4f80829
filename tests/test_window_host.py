"""Plans under a window, and what the calls on windows and shared prefixes refuse (no GPU)."""
import ctypes

import numpy as np
import pytest

from mla_latent_kv_absorb_gb300 import binding

SMS = 152


def parse(image):
    """(clusters' item ranges, items, merge entries) of a plan image."""
    w = [int(x) for x in image]
    clusters, items, combine = w[3], w[4], w[6]
    cl, it, cb = w[7], w[8], w[9]
    return (w[cl:cl + clusters + 1], [w[it + 8 * i:it + 8 * i + 8] for i in range(items)],
            [w[cb + 4 * i:cb + 4 * i + 4] for i in range(combine)])


def seen(L, W, n):
    return {j for j in range(L) if W == 0 or j >= L - W or j < n}


CASES = [([1], 1, 1, 0), ([64, 65, 63], 1, 1, 0), ([300, 7, 1000], 1, 65, 1), ([130], 1, 40, 100), ([128], 1, 64, 64),
         ([129], 1, 64, 64), ([4000], 1, 1, 129), ([2000, 64], 1, 5000, 3), ([6000, 1], 1, 1500, 70), ([100, 250, 1000], 4, 33, 5),
         ([513], 7, 2, 2), ([64] * 200, 1, 64, 0), (list(range(1, 400, 3)), 1, 100, 9), ([100000], 1, 4096, 4)]


@pytest.mark.parametrize("lens,q,W,n", CASES)
@pytest.mark.parametrize("min_pages", [0, 1, 8])
def test_items_read_the_visible_pages_once(lens, q, W, n, min_pages):
    lens = [max(S, q) for S in lens]
    image, info = binding.mla_plan_splits(lens, SMS, queries_per_seq=q, window=W, sinks=n, min_pages_per_split=min_pages)
    ranges, items, combine = parse(image)
    assert info.window == W and info.sinks == n and int(image[15]) == n
    assert ranges[0] == 0 and ranges[-1] == len(items) == info.num_items
    sink_pages = (n + 63) // 64
    got = {}
    for row, begin, end, L, slot, table_row, skip, hole_end in items:
        S = lens[row // q]
        assert table_row == row // q and L == S - q + 1 + row % q and 0 <= begin < end
        assert hole_end == (L - W if L - W > n else 0) and skip >= 0
        for v in range(begin, end):
            page = v if v < sink_pages else v + skip
            tokens = [j for j in range(64 * page, min(64 * page + 64, L)) if not n <= j < hole_end]
            assert tokens, "a page without a visible token"
            got.setdefault(row, []).extend(tokens)
    assert sorted(got) == list(range(len(lens) * q))
    for row, tokens in got.items():
        want = seen(lens[row // q] - q + 1 + row % q, W, n)
        assert len(tokens) == len(want) and set(tokens) == want
    assert info.total_pages == sum(i[2] - i[1] for i in items)
    assert sum(c[2] for c in combine) == info.num_partials


def test_short_windows_use_every_pair():
    _, info = binding.mla_plan_splits([64] * 64, SMS, window=64)
    assert info.num_clusters == 64 and info.num_partials == 0
    # 500 sequences on 76 pairs: some pair has seven, and 72 pairs with at most seven hold them all
    _, info = binding.mla_plan_splits([64] * 500, SMS, window=64)
    assert info.num_clusters == 72 and info.num_partials == 0


def test_without_a_window_plans_are_as_before():
    lens = [100, 5000, 64, 1]
    a, ia = binding.mla_plan_splits(lens, SMS)
    b, ib = binding.mla_plan_splits(lens, SMS, window=0, sinks=0)
    assert np.array_equal(a, b) and ia.num_items == ib.num_items and ia.window == 0
    for item in parse(a)[1]:
        assert item[6:] == [0, 0]


@pytest.mark.parametrize("kw", [dict(window=-1), dict(window=0, sinks=1), dict(window=5, sinks=-1), dict(window=-(2 ** 31))])
def test_plan_refusals(kw):
    with pytest.raises(binding.MlaError) as e:
        binding.mla_plan_splits([100], SMS, **kw)
    assert e.value.status == binding.MLA_ERR_INVALID_ARG


P = 0x10000  # an aligned address that no refused call touches


def window_args(**kw):
    d = dict(dtype=0, pool=P, scale=None, kr=None, pages=9, table=P, max_pages=9, S=500, T=300, W=64, n=4, q_c=P, q_r=P, uk=P, uv=P,
             soft=0.07, ws=P, size=1 << 40, out=P, err=P, stream=None)
    assert not set(kw) - set(d)
    return list({**d, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(W=0), 1), (dict(n=-1), 1), (dict(T=0), 1), (dict(T=501), 1), (dict(S=0), 1), (dict(max_pages=7), 1), (dict(dtype=3), 1),
    (dict(pool=None), 1), (dict(table=None), 1), (dict(q_c=None), 1), (dict(out=None), 1), (dict(err=None), 1), (dict(ws=None), 1),
    (dict(dtype=1), 1), (dict(soft=0.0), 1), (dict(soft=float("nan")), 1), (dict(pool=P + 8), 2), (dict(q_r=P + 8), 2),
    (dict(table=P + 2), 2), (dict(out=P + 4), 2), (dict(size=1000), 4),
    (dict(S=2 ** 31 - 1, T=2 ** 31 - 1, max_pages=2 ** 26, W=2 ** 31 - 1), 3)])
def test_window_chunk_refusals(kw, status):
    assert binding.lib().mla_prefill_window(*window_args(**kw)) == status


def test_window_chunk_workspace():
    f = binding.lib().mla_prefill_window_workspace_bytes
    row = 576 * 2 + 2 * 128 * 128 * 2
    assert f(0, 1, 1, 0) == f(10, 11, 1, 0) == f(10, 5, 0, 0) == f(10, 5, 1, -1) == f(10, 0, 1, 0) == 0
    for S, T, W, n, keys in ((16384, 4096, 1024, 4, 5123), (500, 500, 3, 7, 500), (5000, 1, 1, 0, 1), (5000, 10, 100, 4891, 5000),
                             (5000, 10, 100, 4890, 4999), (2 ** 31 - 1, 1, 1, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert keys * row <= f(S, T, W, n) <= keys * row + 3 * 1024
    with pytest.raises(binding.MlaError):
        binding.mla_prefill_window_workspace_bytes(10, 11, 1)


def attend_args(**kw):
    d = dict(rows=10, P=100, sms=SMS, q_c=P, q_r=P, k=P, v=P, k_r=P, stride=576, soft=0.07, own=P, own_lse=P, ws=P, size=1 << 40, out=P,
             lse=P, err=P, stream=None)
    assert not set(kw) - set(d)
    return list({**d, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(P=0), 1), (dict(sms=0), 1), (dict(soft=-1.0), 1), (dict(soft=float("inf")), 1), (dict(stride=63), 1),
    (dict(stride=2 ** 33), 1), (dict(q_c=None), 1), (dict(k=None), 1), (dict(k_r=None), 1), (dict(own=None), 1), (dict(own_lse=None), 1),
    (dict(ws=None), 1), (dict(out=None), 1), (dict(err=None), 1), (dict(q_c=P + 8), 2), (dict(k_r=P + 2), 2), (dict(stride=68), 2),
    (dict(ws=P + 8), 2), (dict(own=P + 2), 2), (dict(own_lse=P + 2), 2), (dict(lse=P + 1), 2), (dict(rows=65537), 3),
    (dict(P=65535 * 128 + 1), 3), (dict(sms=4097), 3), (dict(size=100), 4), (dict(rows=0, q_c=None), 0)])
def test_prefix_attend_refusals(kw, status):
    assert binding.lib().mla_prefix_attend(*attend_args(**kw)) == status


def test_prefix_workspace():
    f = binding.lib().mla_prefix_attend_workspace_bytes
    assert f(0, 10, SMS) == f(10, 0, SMS) == f(10, 10, 0) == f(65537, 10, SMS) == 0
    # a partial of 128 columns and a log-sum-exp for every row of every segment: workers + runs - 1 of them
    assert f(1, 1, SMS) == (128 + 127) * 129 * 4
    assert f(64, 8192, SMS) == (SMS + 127) * 64 * 129 * 4
    assert f(256, 8192, SMS) == (SMS // 2 + 127) * 256 * 129 * 4
    assert f(257, 8192, SMS) == (SMS // 2 + 255) * 256 * 129 * 4


def open_args(**kw):
    d = dict(dtype=0, pool=P, scale=None, kr=None, pages=9, table=P, max_pages=9, P=500, uk=P, uv=P, rows=P, k=2 * P, v=3 * P, err=P,
             stream=None)
    assert not set(kw) - set(d)
    return list({**d, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(P=0), 1), (dict(P=600), 1), (dict(max_pages=0), 1), (dict(pages=0), 1), (dict(dtype=7), 1), (dict(dtype=2), 1), (dict(pool=None), 1),
    (dict(uk=None), 1), (dict(rows=None), 1), (dict(err=None), 1), (dict(k=P), 1), (dict(v=2 * P), 1), (dict(k=2 * P + 8), 2),
    (dict(uv=P + 4), 2), (dict(table=P + 2), 2), (dict(P=65535 * 128 + 1, max_pages=2 ** 20), 3)])
def test_prefix_open_refusals(kw, status):
    assert binding.lib().mla_prefix_open(*open_args(**kw)) == status


def test_prefix_open_does_not_touch_host_memory():
    """A refused call writes nothing: the arguments above are not mapped, so this process would have ended."""
    assert ctypes.sizeof(binding.PlanOptions) == 32 and ctypes.sizeof(binding.PlanInfo) == 64
