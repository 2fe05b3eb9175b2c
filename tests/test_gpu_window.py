"""Attention within a sliding window and to the first tokens, forward and backward, against
the float64 oracle: element by element within bounds by arithmetic, and as a whole."""
import math

import numpy as np
import pytest
import torch

from cache_util import bf16, np64
from oracle import window

pytestmark = pytest.mark.gpu

U = 2.0 ** -8  # a bf16 rounding, relative


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


def inputs(seed, B, H, Hkv, Lq, Lk, d):
    g = torch.Generator().manual_seed(seed)
    return bf16(g, B, H, Lq, d), bf16(g, B, Hkv, Lk, d), bf16(g, B, Hkv, Lk, d), bf16(g, B, H, Lq, d)


def exact_and_bounds(q, k, v, do, left, right, sinks, scale):
    """{name: (exact, bound)} of o, lse, dq, dk, dv.

    Scores: d products added in fp32, off by d 2^-24 sum |q k| scale, twice for the scaling
    and the base-2 reference; the exponentials 2^-21; sums over n keys n 2^-24: together
    e = the relative error of a weight in fp32. The weights enter the products as bf16 (U).
      O:  (U + 2 e) P |v| twice (the weights and their sum), and its own rounding U |O|
      D:  the sum of |dO| times O's error
      dS: U |dS| for the product, e |dS|, and P times the errors of D and of dP
          (d 2^-24 |dO| |v|); dQ, dK: those times |K|, |Q|, and their rounding
      dV: (U + e) P^T |dO|, and its rounding
    """
    q, k, v, do = (np64(x) for x in (q, k, v, do))
    B, H, Lq, d = q.shape
    Hkv, Lk = k.shape[1:3]
    o, lse = window.forward(q, k, v, left, right, sinks, scale)
    dq, dk, dv = window.backward(q, k, v, do, left, right, sinks, scale)
    seen = window.visible(Lq, Lk, left, right, sinks)
    bo, bl, bq, bk, bv = (np.zeros_like(x) for x in (o, lse, dq, dk, dv))
    n = int(seen.sum(1).max())
    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            Q, K, V, G = q[b, h], k[b, g], v[b, g], do[b, h]
            P, _ = window.weights(Q, K, seen, scale)
            big = float((np.abs(Q) @ np.abs(K).T * seen).max()) * scale
            e = 2 * d * 2.0 ** -24 * big + 2.0 ** -21 + n * 2.0 ** -24
            bo[b, h] = 2 * (U + 2 * e) * (P @ np.abs(V)) + U * np.abs(o[b, h])
            bl[b, h] = e + 2.0 ** -22 * np.where(np.isfinite(lse[b, h]), np.abs(lse[b, h]), 0)
            eD = (np.abs(G) * bo[b, h]).sum(1, keepdims=True) + d * 2.0 ** -24 * (np.abs(G) * np.abs(o[b, h])).sum(1, keepdims=True)
            dP = G @ V.T
            dS = P * (dP - (P * dP).sum(1, keepdims=True))
            w = (U + 2 * e) * np.abs(dS) + P * (eD + d * 2.0 ** -24 * (np.abs(G) @ np.abs(V).T))
            m = H // Hkv * Lq * 2.0 ** -24  # sums over the queries of a group, in fp32
            bq[b, h] = scale * (w + n * 2.0 ** -24 * np.abs(dS)) @ np.abs(K) + U * np.abs(dq[b, h])
            bk[b, g] += scale * (w + m * np.abs(dS)).T @ np.abs(Q)
            bv[b, g] += (U + 2 * e + m) * P.T @ np.abs(G)
    bk += U * np.abs(dk)
    bv += U * np.abs(dv)
    return dict(o=(o, bo), lse=(lse, bl), dq=(dq, bq), dk=(dk, bk), dv=(dv, bv))


def compare(got, want):
    for name, x in got.items():
        x = np64(x)
        ref, bound = want[name]
        blind = np.isneginf(ref)
        assert (np.isneginf(x) == blind).all(), name
        x, ref, bound = x[~blind], ref[~blind], bound[~blind]
        assert np.isfinite(x).all(), name
        assert (np.abs(x - ref) <= bound + 1e-30).all(), (name, np.max(np.abs(x - ref) - bound))
        assert (x[bound == 0] == 0).all()
        # As a whole: at most three independent roundings meet in a value, each of rms U / sqrt(3).
        if ref.size > 4000 and name != "lse" and np.linalg.norm(ref) > 0:
            assert np.linalg.norm(x - ref) <= 2 * U * np.linalg.norm(ref), name


def run(eba, q, k, v, do, left, right, sinks, scale=None, with_rest=True):
    q, k, v, do = (x.cuda() for x in (q, k, v, do))
    o, lse, *rest = eba.fwd_window(q, k, v, left, right, sinks, scale, rest=with_rest)
    need = eba.bwd_window_workspace_size(*q.shape[:2], k.shape[1], q.shape[2], k.shape[2], q.shape[3], left, right, sinks)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN as fp32
    dq, dk, dv = eba.bwd_window(q, k, v, o, do, lse, left, right, sinks, scale, workspace=ws, rest=rest[0] if rest else None)
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


# B, H, H_kv, Lq, Lk, d, left, right, sinks
CASES = [
    (1, 1, 1, 1, 1, 64, 0, 0, 0),
    (2, 2, 1, 1, 1, 128, None, None, 5),
    (1, 2, 2, 5, 5, 64, 1, 0, 1),
    (1, 1, 1, 1, 300, 64, 10, 0, 4),          # one query at the end of many keys
    (1, 2, 1, 300, 1, 128, 10, 0, 0),         # one key: most queries lie before it
    (1, 2, 1, 300, 1, 64, 10, 400, 1),
    (1, 2, 1, 128, 128, 64, None, 0, 0),      # whole tiles
    (1, 2, 2, 129, 129, 128, None, 0, 0),
    (2, 4, 2, 333, 333, 64, 48, 48, 0),
    (1, 3, 1, 257, 400, 128, 100, 0, 3),
    (1, 2, 1, 700, 650, 64, 127, 0, 130),     # sinks beyond a tile, rows that see nothing
    (1, 2, 1, 700, 100, 128, 64, 0, 2),
    (1, 2, 2, 100, 900, 64, 0, 0, 1),         # each query its own key and the first one
    (1, 1, 1, 513, 513, 64, 0, None, 0),      # causal the other way round
    (1, 2, 1, 400, 640, 128, 30, None, 7),
    (1, 2, 2, 384, 384, 64, None, 60, 9),
    (1, 2, 2, 600, 600, 128, 300, 17, 600),   # all are sinks
    (1, 5, 1, 1290, 1290, 64, 60, 0, 4),      # pieces of the first tile's gradients
    (1, 2, 2, 1600, 1600, 128, 33, 20, 200),
    (1, 4, 1, 2100, 2300, 64, 127, 0, 128),
    (2, 3, 3, 520, 520, 128, 128, 0, 0),      # a window of exactly a tile
    (1, 8, 8, 1000, 1000, 64, 255, 256, 1),
    (40, 16, 4, 70, 70, 64, 9, 0, 2),         # many short sequences
    (1, 1, 1, 640, 640, 64, 2**31 - 1, 2**31 - 1, 2**31 - 1),
]


@pytest.mark.parametrize("B,H,Hkv,Lq,Lk,d,left,right,sinks", CASES, ids=lambda x: str(x))
def test_matches_oracle(eba, B, H, Hkv, Lq, Lk, d, left, right, sinks):
    q, k, v, do = inputs(Lq + Lk + d, B, H, Hkv, Lq, Lk, d)
    want = exact_and_bounds(q, k, v, do, left, right, sinks, 1 / math.sqrt(d))
    a, b = run(eba, q, k, v, do, left, right, sinks), run(eba, q, k, v, do, left, right, sinks, with_rest=False)
    compare(a, want)
    compare(b, want)
    assert all(torch.equal(a[n], b[n]) for n in ("o", "lse", "dv"))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left,right", [(1, 0), (2, 2), (7, 0), (30, 30)])
def test_few_keys(eba, left, right, d):
    """O and what its rounding took are the sum in fp32 to bf16 twice; dQ and dK of rows that see
    few keys are then nearer than without: D's error, O's rounding against dO, was the largest."""
    q, k, v, do = inputs(left + d, 2, 4, 4, 300, 300, d)
    want = exact_and_bounds(q, k, v, do, left, right, 0, 1 / math.sqrt(d))
    a, b = run(eba, q, k, v, do, left, right, 0), run(eba, q, k, v, do, left, right, 0, with_rest=False)
    off = lambda x, n: np.linalg.norm(np64(x[n]) - want[n][0]) / np.linalg.norm(want[n][0])  # noqa: E731
    for n in ("dq", "dk"):
        # roundings of dS, of the weights behind D, and of the result: an error that is spread
        # evenly over half a step to both sides has rms U / sqrt(3) of the power of two below
        # its value, three of them together U at most
        assert off(a, n) <= U
    assert off(a, "dq") < off(b, "dq")
    o, lse, rest = eba.fwd_window(*(x.cuda() for x in (q, k, v)), left, right, 0, rest=True)
    assert (rest.float().abs() <= U * o.float().abs() + 1e-38).all()


@pytest.mark.parametrize("seed", range(8))
def test_drawn_sizes(eba, seed):
    r = np.random.default_rng(seed)
    hkv = int(r.integers(1, 4))
    H, d = hkv * int(r.integers(1, 4)), int(r.choice([64, 128]))
    Lq, Lk = (int(x) for x in r.integers(1, 900, 2))
    left, right = (None if r.random() < 0.25 else int(r.integers(0, 500)) for _ in range(2))
    sinks = int(r.choice([0, 1, 4, 140]))
    q, k, v, do = inputs(seed, 1, H, hkv, Lq, Lk, d)
    compare(run(eba, q, k, v, do, left, right, sinks, 0.2), exact_and_bounds(q, k, v, do, left, right, sinks, 0.2))


@pytest.mark.parametrize("d", [64, 128])
def test_long_rows_against_rows_of_their_own(eba, d):
    """12544 tokens: sampled queries against the oracle over the keys they see."""
    L, left, sinks = 12544, 1567, 16
    q, k, v, do = inputs(d, 1, 2, 1, L, L, d)
    got = run(eba, q, k, v, do, left, 0, sinks)
    scale = 1 / math.sqrt(d)
    for i in (0, 15, 16, 127, 128, 1583, 1584, 6000, 12543):
        mine = [j for j in range(i + 1) if j >= i - left or j < sinks]
        args = [x[:, :, s] for x, s in ((q, [i]), (k, mine), (v, mine), (do, [i]))]
        want = exact_and_bounds(*args, None, None, 0, scale)
        compare(dict(o=got["o"][:, :, [i]], lse=got["lse"][:, :, [i]], dq=got["dq"][:, :, [i]]), want)


def test_no_ends_is_plain_attention(eba):
    q, k, v, do = inputs(3, 2, 4, 2, 500, 500, 64)
    got = run(eba, q, k, v, do, None, None, 0, with_rest=False)
    o, lse = eba.fwd(q.cuda(), k.cuda(), v.cuda())
    assert (got["o"] == o).all() and (got["lse"] == lse).all()
    _, dk, dv = eba.bwd(q.cuda(), k.cuda(), v.cuda(), o, do.cuda(), lse)
    assert (got["dk"] == dk).all() and (got["dv"] == dv).all()


def test_hidden_values_do_not_reach(eba):
    """Finite values of any size where they are not seen change nothing, bit for bit."""
    q, k, v, do = inputs(4, 1, 2, 2, 600, 600, 64)
    a = run(eba, q, k, v, do, 100, 0, 2)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 300:], v2[:, :, 300:] = 1e30, -1e30
    b = run(eba, q, k2, v2, do, 100, 0, 2)
    for n in ("o", "lse"):
        assert (a[n][:, :, :300] == b[n][:, :, :300]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_leave_no_weight(eba, d):
    """Scores of -inf everywhere a row sees (O = 0, lse = -inf), and very sharp rows."""
    q, k, v, do = inputs(5, 1, 1, 1, 300, 300, d)
    q[:, :, 7] = 3e38
    k[:, :, :9] = -3e38
    got = eba.fwd_window(q.cuda(), k.cuda(), v.cuda(), 4, 0, 0)
    assert (got[0][:, :, 7] == 0).all() and torch.isneginf(got[1][:, :, 7]).all()
    q, k, v, do = inputs(6, 1, 2, 2, 300, 300, d)
    compare(run(eba, q, k, v, do, 50, 3, 2, 2.0), exact_and_bounds(q, k, v, do, 50, 3, 2, 2.0))


def test_autograd(eba):
    q, k, v, do = (x.cuda() for x in inputs(7, 2, 4, 2, 333, 333, 64))
    for x in (q, k, v):
        x.requires_grad_(True)
    o = eba.attention_window(q, k, v, 40, 0, 3)
    dq, dk, dv = torch.autograd.grad(o, (q, k, v), do.transpose(1, 2).contiguous().transpose(1, 2))
    o2, lse, rest = eba.fwd_window(q.detach(), k.detach(), v.detach(), 40, 0, 3, rest=True)
    _, dk2, dv2 = eba.bwd_window(q.detach(), k.detach(), v.detach(), o2, do, lse, 40, 0, 3, rest=rest)
    assert (o == o2).all() and (dk == dk2).all() and (dv == dv2).all()
    # an expanded gradient, a frozen input, a graph of the gradient
    k2 = k.detach()
    o = eba.attention_window(q, k2, v, 40, 0, 3)
    o.sum().backward()
    assert k2.grad is None and q.grad is not None and v.grad is not None
    one = torch.ones_like(do)
    g = eba.bwd_window(q.detach(), k2, v.detach(), o2, one, lse, 40, 0, 3)
    assert (v.grad == g[2]).all()
    o = eba.attention_window(q, k, v, 40, 0, 3)
    (dq,) = torch.autograd.grad(o, (q,), do, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dq.float().sum(), (q,))


def test_captured_training_step(eba):
    q, k, v, do = (x.cuda() for x in inputs(8, 1, 4, 2, 1200, 1200, 128))
    args = [x.clone().requires_grad_(True) for x in (q, k, v)]

    def step():
        o = eba.attention_window(*args, 90, 0, 4)
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
    for seed in (21, 22):
        new = [x.cuda() for x in inputs(seed, 1, 4, 2, 1200, 1200, 128)]
        with torch.no_grad():
            for a, x in zip(args, new):
                a.copy_(x)
        do.copy_(new[3])
        graph.replay()
        torch.cuda.synchronize()
        want = run(eba, *(x.cpu() for x in new), 90, 0, 4)
        assert (out[0] == want["o"]).all() and (out[2] == want["dk"]).all() and (out[3] == want["dv"]).all()
        # dQ is added up in any order, so that a sum next to a border of two bf16 numbers may
        # take either: one half step in few elements, here below one in 256 of them
        dq = np64(want["dq"])
        assert np.linalg.norm(np64(out[1]) - dq) <= 2 * U / 16 * np.linalg.norm(dq)


def test_refusals(eba):
    q, k, v, do = (x.cuda() for x in inputs(9, 1, 2, 2, 70, 70, 64))
    o, lse = eba.fwd_window(q, k, v, 5)
    for bad in (dict(left=-1), dict(left=5, right=-2), dict(left=5, sinks=-1), dict(left=5.0)):
        with pytest.raises(ValueError):
            eba.fwd_window(q, k, v, **bad)
        with pytest.raises(ValueError):
            eba.bwd_window(q, k, v, o, do, lse, **bad)
    with pytest.raises(ValueError):
        eba.fwd_window(q, k.transpose(1, 2), v, 5)
    with pytest.raises(ValueError):
        eba.bwd_window(q, k, v, o, do[:, :, :69], lse, 5)
    with pytest.raises(ValueError):
        eba.bwd_window(q, k, v, o, do, lse, 5, rest=o.float())
    with pytest.raises(ValueError):
        eba.bwd_window(q, k, v, o, do, lse, 5, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("left,right,sinks", [(100, 50, 0), (130, 0, 3), (0, 200, 0)])
def test_heads_beyond_l2(eba, left, right, sinks):
    """More heads than are walked side by side: the same bits as each batch alone."""
    q, k, v, do = (x.cuda() for x in inputs(31, 4, 128, 128, 300, 300, 128))
    o, lse = eba.fwd_window(q, k, v, left, right, sinks)
    dq, dk, dv = eba.bwd_window(q, k, v, o, do, lse, left, right, sinks)
    for b in range(4):
        one = [x[b:b + 1] for x in (q, k, v)]
        o1, lse1 = eba.fwd_window(*one, left, right, sinks)
        dq1, dk1, dv1 = eba.bwd_window(*one, o1, do[b:b + 1], lse1, left, right, sinks)
        for x, y in ((o, o1), (lse, lse1), (dk, dk1), (dv, dv1)):
            assert torch.equal(x[b:b + 1], y)
        assert (dq[b:b + 1].float() - dq1.float()).norm() <= 2 * U / 16 * dq1.float().norm()


def test_two_steps_at_once(eba):
    """Training steps on streams of their own, at the same time."""
    steps = []
    for seed, (L, d, left, right) in enumerate(((823, 128, 100, 5), (1500, 64, 40, 0), (640, 128, 600, None))):
        q, k, v, do = (x.cuda() for x in inputs(seed, 1, 8, 4, L, L, d))
        for x in (q, k, v):
            x.requires_grad_(True)
        steps.append(((q, k, v), do, (left, right, 2)))

    def step(args, do, window):
        o = eba.attention_window(*args, *window)
        return (o.detach(), *torch.autograd.grad(o, args, do))

    alone = [step(*s) for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    got = [[] for _ in steps]
    for _ in range(10):
        for s, stream, out in zip(steps, streams, got):
            with torch.cuda.stream(stream):
                out.append(step(*s))
    torch.cuda.synchronize()
    for want, outs in zip(alone, got):
        for x in outs:
            # (dq is added up in any order: see test_captured_training_step)
            assert all(torch.equal(want[i], x[i]) for i in (0, 2, 3))
            assert (want[1].float() - x[1].float()).norm() <= 2 * U / 16 * want[1].float().norm()
