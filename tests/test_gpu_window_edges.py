"""Windowed attention where its masks leave nothing or hide something: rows without a weight,
hidden values of any finite size, NaN where no pair of a tile is visible."""
import math

import numpy as np
import pytest
import torch

from cache_util import np64
from test_gpu_window import U, compare, exact_and_bounds, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eba():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


@pytest.fixture(autouse=True)
def status_is_clean(eba):
    eba.poll_device_status()
    yield
    assert eba.poll_device_status() == 0


@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_row_without_a_weight_has_no_gradients(eba, d, H, Hkv):
    """All that row 7 sees has the score -inf: its weights are 0, so it gets no gradient and adds
    none, as if its dO were 0."""
    q, k, v, do = inputs(5, 1, H, Hkv, 300, 300, d)
    k[:, :, 3:8] = -1
    q[:, :, 7], do7 = 0, do[:, :, 7].clone()
    do[:, :, 7] = 0
    want = exact_and_bounds(q, k, v, do, 4, 0, 0, 1 / math.sqrt(d))
    q[:, :, 7], do[:, :, 7] = 3e38, do7
    for with_rest in (True, False):
        got = run(eba, q, k, v, do, 4, 0, 0, with_rest=with_rest)
        assert (got["o"][:, :, 7] == 0).all() and torch.isneginf(got["lse"][:, :, 7]).all()
        assert (got["dq"][:, :, 7] == 0).all()
        others = [i for i in range(300) if i != 7]
        rows = {n: got[n] if n in ("dk", "dv") else got[n][:, :, others] for n in got}
        compare(rows, {n: want[n] if n in ("dk", "dv") else tuple(x[:, :, others] for x in want[n]) for n in want})


@pytest.mark.parametrize("size", [1e30, 3e38])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_values_do_not_reach_gradients(eba, d, H, Hkv, size):
    """Keys and values from 300 on of any finite size: rows that do not see them, and keys that
    only such rows see, keep their gradients (dQ but for the order in which it is added up)."""
    q, k, v, do = inputs(4, 1, H, Hkv, 600, 600, d)
    a = run(eba, q, k, v, do, 100, 0, 2)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 300:], v2[:, :, 300:] = size, -size
    b = run(eba, q, k2, v2, do, 100, 0, 2)
    for n in ("o", "lse"):
        assert torch.equal(a[n][:, :, :300], b[n][:, :, :300])
    for n in ("dk", "dv"):  # (keys 0 and 1 are seen by all rows)
        assert torch.equal(a[n][:, :, 2:200], b[n][:, :, 2:200]), n
    x, y = np64(a["dq"][:, :, :300]), np64(b["dq"][:, :, :300])
    assert np.isfinite(y).all() and np.linalg.norm(x - y) <= 2 * U / 16 * np.linalg.norm(x)


@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_that_no_query_sees(eba, d, H, Hkv):
    """Key tiles without a visible pair: NaN there reaches nothing, and their gradients are 0
    whatever the queries are."""
    q, k, v, do = inputs(11, 1, H, Hkv, 300, 1200, d)  # places 900 to 1199: tiles from 896 on
    a = run(eba, q, k, v, do, 3, 0, 0)
    k[:, :, :896], v[:, :, :896] = math.nan, math.nan
    b = run(eba, q, k, v, do, 3, 0, 0)
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n
    assert (b["dk"][:, :, :896] == 0).all() and (b["dv"][:, :, :896] == 0).all()
    x, y = np64(a["dq"]), np64(b["dq"])
    assert np.isfinite(y).all() and np.linalg.norm(x - y) <= 2 * U / 16 * np.linalg.norm(x)
    q[:, :, 5], do[:, :, 5] = math.nan, math.nan
    c = run(eba, q, k, v, do, 3, 0, 0)
    assert (c["dk"][:, :, :896] == 0).all() and (c["dv"][:, :, :896] == 0).all()


@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk,nan", [(700, 100, 512), (2600, 300, 2176)])
def test_queries_that_see_no_key(eba, Lq, Lk, nan, d, H, Hkv):
    """Query tiles before the first key: NaN there reaches no gradient. (The second case: also
    where the first tokens' gradients are cut in pieces.)"""
    q, k, v, do = inputs(12, 1, H, Hkv, Lq, Lk, d)
    a = run(eba, q, k, v, do, 64, 0, 4)
    q[:, :, :nan], do[:, :, :nan] = math.nan, math.nan
    b = run(eba, q, k, v, do, 64, 0, 4)
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n
    x, y = np64(a["dq"]), np64(b["dq"])
    assert (y[:, :, :Lq - Lk] == 0).all()
    assert np.isfinite(y).all() and np.linalg.norm(x - y) <= 2 * U / 16 * np.linalg.norm(x)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk", [(300, 172), (200, 100), (556, 300)])
def test_rows_that_see_nothing_are_zero_beside_nan(eba, Lq, Lk, d):
    """Rows without a key give O = 0 also where others of their tiles see a NaN value."""
    q, k, v, do = inputs(13, 3, 4, 2, Lq, Lk, d)
    v[:, :, 0] = math.nan
    o, lse, rest = eba.fwd_window(*(x.cuda() for x in (q, k, v)), 20, 0, 0, rest=True)
    blind = Lq - Lk
    assert (o[:, :, :blind] == 0).all() and (rest[:, :, :blind] == 0).all()
    assert torch.isneginf(lse[:, :, :blind]).all()
    assert torch.isnan(o[:, :, blind:blind + 21]).all() and torch.isfinite(lse[:, :, blind:]).all()
    got = run(eba, q, k, v, do, 20, 0, 0)
    assert (got["dq"][:, :, :blind] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_nan_that_is_seen_shows(eba, d):
    """A NaN query or a NaN key makes the rows that see it NaN, o and lse."""
    q, k, v, _ = inputs(14, 1, 2, 2, 400, 400, d)
    q[:, 0, 30] = math.nan
    k[:, 1, 50] = math.nan
    o, lse, rest = eba.fwd_window(*(x.cuda() for x in (q, k, v)), 10, 0, 0, rest=True)
    assert torch.isnan(o[:, 0, 30]).all() and torch.isnan(lse[:, 0, 30]).all()
    assert torch.isnan(o[:, 1, 50:61]).all() and torch.isnan(lse[:, 1, 50:61]).all()
    others = [i for i in range(400) if i != 30]
    assert torch.isfinite(o[:, 0, others]).all() and torch.isfinite(lse[:, 0, others]).all()
    rest_of = [i for i in range(400) if not 50 <= i <= 60]
    assert torch.isfinite(o[:, 1, rest_of]).all() and torch.isfinite(lse[:, 1, rest_of]).all()


@pytest.mark.parametrize("H,Hkv,sinks", [(160, 160, 4), (320, 160, 4), (80, 80, 200)])
@pytest.mark.parametrize("d", [64, 128])
def test_sinks_of_many_heads_stay_whole(eba, d, H, Hkv, sinks):
    """More than 608 key tiles of sinks together are no longer cut in pieces, as those of a batch
    alone are: both against the oracle, for some heads of each batch."""
    L, left = 1200, 60
    q, k, v, do = inputs(15, 4, H, Hkv, L, L, d)
    plain = [eba.bwd_workspace_size(B, H, L, L, d) for B in (1, 4)]
    need = [eba.bwd_window_workspace_size(B, H, Hkv, L, L, d, left, 0, sinks) for B in (1, 4)]
    assert need[0] > plain[0] and need[1] == plain[1]
    together = run(eba, q, k, v, do, left, 0, sinks)
    alone = run(eba, *(x[2:3] for x in (q, k, v, do)), left, 0, sinks)
    for b, g in ((0, 0), (2, Hkv // 2), (3, Hkv - 1)):
        heads = slice(g * H // Hkv, (g + 1) * H // Hkv)
        want = exact_and_bounds(q[b:b + 1, heads], k[b:b + 1, g:g + 1], v[b:b + 1, g:g + 1], do[b:b + 1, heads], left, 0,
                                sinks, 1 / math.sqrt(d))
        for got, at in ((together, b), (alone, 0)) if b == 2 else ((together, b),):
            compare({n: x[at:at + 1, g:g + 1] if n in ("dk", "dv") else x[at:at + 1, heads] for n, x in got.items()}, want)


def test_captured_step_with_unseen_keys(eba):
    """The zeros of keys that no query sees are part of a captured call."""
    q, k, v, do = (x.cuda() for x in inputs(16, 2, 4, 2, 300, 1200, 128))
    args = [x.clone().requires_grad_(True) for x in (q, k, v)]

    def step():
        o = eba.attention_window(*args, 60, 0, 4)
        return (o, *torch.autograd.grad(o, args, do))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for x in out[2:]:
            x.detach().fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want = run(eba, *(x.cpu() for x in (q, k, v, do)), 60, 0, 4)
        assert torch.equal(out[0], want["o"]) and torch.equal(out[2], want["dk"]) and torch.equal(out[3], want["dv"])
        assert (out[2][:, :, 128:768] == 0).all()


@pytest.mark.parametrize("Lq,Lk,left,right,sinks", [(1, 1, None, 0, 1), (1, 1, 1, 0, 0), (300, 1, 10, 0, 0), (300, 1, None, 400, 5),
                                                    (1, 700, 0, 0, 0), (1, 700, 0, 5, 0), (500, 500, 0, 0, 0), (260, 900, 0, 0, 0),
                                                    (900, 260, 0, 0, 0)])
@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (10, 2, 128)])
def test_one_key_a_row_has_no_gradient_but_its_values(eba, Lq, Lk, left, right, sinks, H, Hkv, d):
    """A softmax of one score is 1: dQ and dK are 0, not what rounding leaves."""
    q, k, v, do = inputs(Lq + Lk, 2, H, Hkv, Lq, Lk, d)
    got = run(eba, q, k, v, do, left, right, sinks)
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()
    want = exact_and_bounds(q, k, v, do, left, right, sinks, 1 / math.sqrt(d))
    assert np.abs(want["dq"][0]).max() < 1e-12
    compare({n: got[n] for n in ("o", "lse", "dv")}, want)
