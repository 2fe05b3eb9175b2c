"""Rotary positions (forward, gradient) and the cache append against the float64
oracle, and the operators together: rotation, attention and their gradients;
prompt and tokens through the cache."""
import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import E4M3, Paged, bf16, np64, rope_exact, rope_tolerance

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


def close(got, x, pos, plan, inverse=False):
    """got against the exact rotation of x, both [T, H, d]."""
    exact = rope_exact(np64(x), pos, plan, inverse)
    err, tol = np.abs(np64(got) - exact), rope_tolerance(x, exact, plan)
    assert (err <= tol).all(), np.max(err - tol)


# tokens, H, H_k, d, axes, pairing, positions below
ROPES = [
    (1, 1, 0, 64, (32,), "half", 10),
    (1, 3, 1, 128, (64,), "interleaved", 2 ** 31 - 1),
    (7, 5, 5, 64, (8, 12, 12), "half", 100),
    (33, 8, 2, 128, (20, 22, 22), "interleaved", 10 ** 6),
    (130, 2, 1, 128, (1, 2, 5), "half", 50),           # 16 of 128 elements turn
    (130, 2, 1, 64, (3, 5, 7, 9), "interleaved", 5000),  # 48 of 64; four axes
    (1000, 4, 4, 64, (16,), "half", 10 ** 8),
    (5000, 9, 3, 128, (10, 11, 35), "half", 3000),       # an odd number of heads
]


@pytest.mark.parametrize("T,H,Hk,d,axes,pairing,far", ROPES, ids=lambda x: str(x).replace(" ", ""))
def test_rope_matches_oracle(eba, T, H, Hk, d, axes, pairing, far):
    g = torch.Generator().manual_seed(T + H + d)
    q, k = bf16(g, T, H, d), (bf16(g, T, Hk, d) if Hk else None)
    pos = torch.randint(-far, far, (len(axes), T), generator=g).to(torch.int32)
    plan = eba.Rope(axes, pairing=pairing)
    gk = None if k is None else k.cuda()
    for fn, inverse in ((eba.rope_fwd, False), (eba.rope_bwd, True)):
        qo, ko = fn(q.cuda(), gk, pos.cuda(), plan)
        close(qo, q, pos, plan, inverse)
        if Hk:
            close(ko, k, pos, plan, inverse)
        else:
            assert ko is None
        if len(axes) == 1:
            assert torch.equal(fn(q.cuda(), gk, pos[0].cuda(), plan)[0], qo)


def test_the_first_and_the_last_position(eba):
    # position 0 leaves the head as it is; the largest and smallest int32 are as
    # exact as any other
    plan = eba.Rope((64,))
    x = bf16(torch.Generator().manual_seed(1), 4, 2, 128)
    pos = torch.tensor([0, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32)
    got, _ = eba.rope_fwd(x.cuda(), None, pos.cuda(), plan)
    assert torch.equal(got[0].cpu(), x[0])
    close(got, x, pos[None], plan)


def test_own_frequencies(eba):
    freq = [0.0, 1.0, -1.0, 7.5, 2 * math.pi, 100.0, 1e-9, 0.25]
    plan = eba.Rope((3, 5), frequencies=freq)
    x = bf16(torch.Generator().manual_seed(2), 50, 2, 64)
    pos = torch.randint(-10 ** 6, 10 ** 6, (2, 50), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    got, _ = eba.rope_fwd(x.cuda(), None, pos.cuda(), plan)
    close(got, x, pos, plan)
    assert torch.equal(got[..., 16:].cpu(), x[..., 16:])  # behind the rotated elements
    assert torch.equal(got[..., 0].cpu(), x[..., 0])      # frequency 0


@pytest.mark.parametrize("d,axes", [(64, (8, 12, 12)), (128, (64,))])
def test_layouts_views_and_shared_positions(eba, d, axes):
    B, H, Hk, L = 3, 6, 2, 37
    g = torch.Generator().manual_seed(4)
    plan = eba.Rope(axes)
    q, k = bf16(g, B, H, L, d).cuda(), bf16(g, B, Hk, L, d).cuda()
    shared = torch.randint(0, 9999, (len(axes), L), generator=g).to(torch.int32).cuda()
    own = torch.randint(0, 9999, (len(axes), B, L), generator=g).to(torch.int32).cuda()
    for pos in (shared, own):
        qo, ko = eba.rope_fwd(q, k, pos, plan)
        assert qo.is_contiguous() and qo.shape == q.shape
        for b in range(B):
            pb = pos if pos.dim() == 2 else pos[:, b]
            close(qo[b].transpose(0, 1), q[b].transpose(0, 1), pb.cpu(), plan)
            close(ko[b].transpose(0, 1), k[b].transpose(0, 1), pb.cpu(), plan)
    # views: the three parts of one projection, a transposed layout, an expanded k
    qkv = bf16(g, L, H + 2 * Hk, d).cuda()
    qv, kv = qkv[:, :H], qkv[:, H:H + Hk]
    a = eba.rope_fwd(qv, kv, shared, plan)
    b = eba.rope_fwd(qv.contiguous(), kv.contiguous(), shared, plan)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    t = q.transpose(1, 2).contiguous().transpose(1, 2)  # token-major memory
    assert torch.equal(eba.rope_fwd(t, None, own, plan)[0], eba.rope_fwd(q, None, own, plan)[0])
    one = k[:, :1].expand(B, H, L, d)
    assert torch.equal(eba.rope_fwd(q, one, own, plan)[1], eba.rope_fwd(q, one.contiguous(), own, plan)[1])


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_autograd_is_the_transpose(eba, pairing):
    # <R x, g> = <x, R^T g>: the rotation is linear, so this is its difference
    # quotient in every direction at once; bf16 roundings of R x and R^T g are
    # random, 2^-8 each at most over 2 sums of N terms
    g = torch.Generator().manual_seed(5)
    plan = eba.Rope((8, 12, 12), pairing=pairing)
    q, k = bf16(g, 40, 4, 64).cuda().requires_grad_(), bf16(g, 40, 2, 64).cuda().requires_grad_()
    pos = torch.randint(0, 500, (3, 40), generator=g).to(torch.int32)
    gq, gk = bf16(g, 40, 4, 64).cuda(), bf16(g, 40, 2, 64).cuda()
    qo, ko = eba.rope(q, k, pos.cuda(), plan)
    dq, dk = torch.autograd.grad((qo, ko), (q, k), (gq, gk))
    for x, y, grad, dx in ((q, qo, gq, dq), (k, ko, gk, dk)):
        close(dx, grad, pos, plan, inverse=True)
        a, b = (np64(y) * np64(grad)).sum(), (np64(x) * np64(dx)).sum()
        assert abs(a - b) <= 2.0 ** -8 * (np.abs(np64(y) * np64(grad)).sum() + np.abs(np64(x) * np64(dx)).sum())
    # one output alone, an expanded gradient (a sum's), and a transposed one
    qo, ko = eba.rope(q, k, pos.cuda(), plan)
    dk, = torch.autograd.grad(ko.sum(), k)
    close(dk, torch.ones_like(k), pos, plan, inverse=True)
    qo, _ = eba.rope(q, None, pos.cuda(), plan)
    w = bf16(g, 64, 4, 40).cuda().permute(2, 1, 0)
    dq, = torch.autograd.grad(qo, q, w)
    close(dq, w, pos, plan, inverse=True)
    # and the gradient's gradient is the rotation again
    gq2 = gq.clone().requires_grad_()
    dq, = torch.autograd.grad(eba.rope(q, None, pos.cuda(), plan)[0], q, gq2, create_graph=True)
    back, = torch.autograd.grad(dq, gq2, gq)
    close(back, gq, pos, plan)


def test_rotation_captured_forward_and_backward(eba):
    g = torch.Generator().manual_seed(6)
    plan = eba.Rope((32,))
    q = bf16(g, 64, 2, 64).cuda().requires_grad_()
    gq = bf16(g, 64, 2, 64).cuda()
    pos = torch.arange(64, device="cuda", dtype=torch.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(eba.rope(q, None, pos, plan)[0], q, gq)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = eba.rope(q, None, pos, plan)
        dq, = torch.autograd.grad(y, q, gq)
    with torch.no_grad():
        q.copy_(q.flip(0))
        pos.add_(1000)
    graph.replay()
    close(y, q, pos[None].cpu(), plan)
    close(dq, gq, pos[None].cpu(), plan, inverse=True)


def test_rotation_and_attention_trained_together(eba):
    # grouped heads, three axes: gradients of sum(O dO) with respect to the
    # unrotated q and k against the exact ones. The attention's own bar for
    # bf16 inputs is 2e-2 on unit-variance data; the rotations before and behind
    # it add half a bf16 step each, 2^-8 of values below 4.
    B, H, Hk, L, d = 1, 4, 2, 200, 64
    g = torch.Generator().manual_seed(7)
    q, k, v, do = bf16(g, B, H, L, d), bf16(g, B, Hk, L, d), bf16(g, B, Hk, L, d), bf16(g, B, H, L, d)
    plan = eba.Rope((8, 12, 12))
    pos = torch.stack([torch.arange(L) // 49, torch.arange(L) // 7 % 7, torch.arange(L) % 7]).to(torch.int32)
    gq, gk, gv = (x.cuda().requires_grad_() for x in (q, k, v))
    o = eba.attention(*eba.rope(gq, gk, pos.cuda(), plan), gv)
    o.backward(do.cuda())

    def turn(x, inverse=False):
        return np.stack([rope_exact(y.swapaxes(0, 1), pos, plan, inverse).swapaxes(0, 1) for y in x])

    rq, rk, scale = turn(np64(q)), turn(np64(k)), 1 / math.sqrt(d)
    ro, _ = oracle.gqa_forward(rq, rk, np64(v), scale)
    dq, dk, dv = oracle.gqa_backward(rq, rk, np64(v), np64(do), scale)
    for got, exact in ((o, ro), (gq.grad, turn(dq, True)), (gk.grad, turn(dk, True)), (gv.grad, dv)):
        assert np.abs(np64(got) - exact).max() <= 2e-2 + 2 * 2.0 ** -8 * 4


# ---------------------------------------------------------------------------
# The append
# ---------------------------------------------------------------------------

def append_case(eba, lens, new, H, d, page, *, e4m3=False, heads_first=False, axes=None,
                pairing="half", positions=True, padding=0, seed=0):
    """Appends the last new[b] tokens of each sequence and checks every slot of the
    cache: the new rows against the oracle, all others bit for bit as before."""
    sc = dict(k_scale=0.02, v_scale=0.25) if e4m3 else {}
    p = Paged(lens, page, H, d, e4m3=e4m3, heads_first=heads_first, seed=seed, **sc)
    cache = p.on_gpu(eba)
    before = [t.view(torch.uint8).clone() for t in (p.gk, p.gv)]
    T = sum(new) + padding
    g = torch.Generator().manual_seed(seed + 1)
    k, v = bf16(g, T, H, d), bf16(g, T, H, d)
    one_each = all(n == 1 for n in new) and not padding
    cu = None
    if not one_each:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    plan = pos = None
    if axes:
        plan = eba.Rope(axes, pairing=pairing)
        pos = torch.randint(-5, 10 ** 6, (len(axes), T), generator=g).to(torch.int32)
    eba.cache_append(cache, k.cuda(), v.cuda(), p.gtable, p.glens, cu, rope=plan,
                     positions=pos.cuda() if axes and positions else None)
    place = np.full(T, 0)
    t = 0
    for b, n in enumerate(new):
        place[t:t + n] = np.arange(lens[b] - n, lens[b])
        t += n
    ek = np64(k)
    if axes:
        ek = rope_exact(ek, pos if positions else place[None], plan)
        tk = rope_tolerance(k, ek, plan)
    else:
        tk = np.zeros_like(ek)
    got_k, got_v = np64(p.pages(p.gk)), np64(p.pages(p.gv))
    changed = np.zeros(got_k.shape[:2], bool)
    t = 0
    for b, n in enumerate(new):
        for i in range(n):
            if lens[b]:
                page_, slot = p.rows[b][place[t] // page], place[t] % page
                changed[page_, slot] = True
                for got, exact, scale, tol in ((got_k[page_, slot], ek[t], p.k_scale, tk[t]),
                                               (got_v[page_, slot], np64(v[t]), p.v_scale, 0)):
                    if e4m3:
                        # half a step, 2^-4 of the value and 2^-10 among the
                        # smallest, on top of the fp32 rotation and scaling
                        want = np.clip(exact / np.float64(np.float32(scale)), -448, 448)
                        fine = 2.0 ** -19 * (np.abs(want) + 4 / scale)
                        assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + fine).all()
                    else:
                        assert (np.abs(got - exact) <= tol).all()
            t += 1
    keep = torch.tensor(~changed)
    for now, was in zip((p.gk, p.gv), before):
        assert torch.equal(p.pages(now.view(torch.uint8)).cpu()[keep], p.pages(was).cpu()[keep])


APPENDS = [
    ([1], [1], 1, 64, 16, {}),
    ([5], [5], 3, 128, 4, dict(axes=(64,))),
    ([40, 17, 64, 100], [1, 1, 1, 1], 8, 128, 16, dict(axes=(20, 22, 22), pairing="interleaved")),
    ([40, 0, 64, 0], [1, 1, 1, 1], 2, 64, 7, dict(axes=(32,), positions=False)),   # empty slots
    ([300, 20, 77], [250, 0, 77], 2, 64, 16, dict(axes=(8, 12, 12))),
    ([300, 20, 77], [250, 3, 60], 5, 128, 48, dict(padding=9)),                     # rows behind the last
    ([33, 129], [33, 100], 4, 64, 16, dict(e4m3=True, axes=(8,), padding=1)),
    ([90, 70], [1, 1], 2, 128, 32, dict(e4m3=True, heads_first=True, axes=(64,), positions=False)),
    ([700, 650], [700, 3], 16, 64, 33, dict(heads_first=True, axes=(16, 16), pairing="interleaved")),
    ([4000], [3999], 8, 128, 16, dict(e4m3=True, axes=(64,), positions=False)),
]


@pytest.mark.parametrize("lens,new,H,d,page,kw", APPENDS, ids=lambda x: str(x).replace(" ", ""))
def test_append_matches_oracle(eba, lens, new, H, d, page, kw):
    append_case(eba, lens, new, H, d, page, seed=sum(lens), **kw)


def test_append_offsets_that_begin_behind_the_first_rows(eba):
    p = Paged([20, 9], 8, 2, 64, seed=41)
    cache = p.on_gpu(eba)
    k = bf16(torch.Generator().manual_seed(1), 10, 2, 64).cuda()
    before = p.gk.clone()
    eba.cache_append(cache, k, k, p.gtable, p.glens, torch.tensor([3, 5, 6], device="cuda", dtype=torch.int32))
    rows = {(p.rows[0][2], 2): 3, (p.rows[0][2], 3): 4, (p.rows[1][1], 0): 5}
    for (page, slot), t in rows.items():
        assert torch.equal(p.gk[page, slot], k[t]) and torch.equal(p.gv[page, slot], k[t])
        before[page, slot] = k[t]
    assert torch.equal(p.gk.view(torch.uint8), before.view(torch.uint8))


def test_positions_shared_by_the_axes(eba):
    plan = eba.Rope((16, 16))
    x = bf16(torch.Generator().manual_seed(2), 30, 3, 64).cuda()
    pos = torch.arange(30, device="cuda", dtype=torch.int32)
    both = pos.expand(2, 30)  # a stride of 0
    assert torch.equal(eba.rope_fwd(x, None, both, plan)[0], eba.rope_fwd(x, None, both.contiguous(), plan)[0])


def test_append_to_hundreds_of_sequences(eba):
    r = np.random.default_rng(1)
    new = [int(x) for x in r.integers(0, 6, size=300)]
    lens = [n + int(x) for n, x in zip(new, r.integers(0, 30, size=300))]
    append_case(eba, lens, new, 2, 64, 16, axes=(32,), padding=5, seed=8)


def test_append_e4m3_saturates_and_keeps_nan(eba):
    p = Paged([4], 4, 1, 64, e4m3=True)
    cache = p.on_gpu(eba)
    k = torch.zeros(1, 1, 64)
    k[0, 0, :5] = torch.tensor([1000.0, -math.inf, math.nan, math.inf, 2.0 ** -11])
    eba.cache_append(cache, k.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda(), p.gtable, p.glens)
    for t in (p.gk, p.gv):
        got = np64(t[p.rows[0][0], 3, 0])
        assert got[0] == 448 and got[1] == -448 and np.isnan(got[2]) and got[3] == 448 and got[4] == 0


def test_append_reports_bad_places(eba):
    p = Paged([20, 20, 20, 20], 16, 1, 64)
    cache = p.on_gpu(eba)
    before = p.gk.view(torch.uint8).clone()
    k = bf16(torch.Generator().manual_seed(1), 8, 1, 64).cuda()
    table, lens = p.gtable.clone(), p.glens.clone()
    table[0, 1], table[1, 1] = p.n_pages, -1  # pages that are none
    lens[2], lens[3] = 1, 16 * table.shape[1] + 2  # fewer than the new tokens; behind the table
    cu = torch.tensor([0, 2, 4, 6, 8], device="cuda", dtype=torch.int32)
    eba.cache_append(cache, k, k, table, lens, cu)
    assert eba.poll_device_status() == 7
    page, slot = p.rows[2][0], 0  # the one token that has a place
    assert torch.equal(p.gk[page, slot], k[5])
    after = p.gk.view(torch.uint8).clone()
    after[page, slot] = before[page, slot]
    assert torch.equal(after, before)


def test_append_with_offsets_that_decrease_writes_in_no_other_place(eba):
    p = Paged([20, 20, 20], 16, 1, 64)
    cache = p.on_gpu(eba)
    held = torch.zeros((p.n_pages, 16), dtype=torch.bool)
    for r in p.rows:  # the places of tokens
        held[r[0]], held[r[1], :4] = True, True
    before = p.gk.view(torch.uint8).clone()
    k = bf16(torch.Generator().manual_seed(1), 6, 1, 64).cuda()
    for cu in ([0, 5, 1, 6], [0, 2, -3, 6], [3, 0, 0, 6], [0, 2 ** 31 - 1, -2 ** 31, 6]):
        eba.cache_append(cache, k, k, p.gtable, p.glens, torch.tensor(cu, device="cuda", dtype=torch.int32))
    eba.poll_device_status()
    assert torch.equal(p.gk.view(torch.uint8).cpu()[~held], before.cpu()[~held])


def test_append_from_one_projection_and_captured(eba):
    p = Paged([64, 70], 16, 2, 64, seed=4)
    q = Paged([64, 70], 16, 2, 64, seed=4)
    qkv = bf16(torch.Generator().manual_seed(2), 2, 12, 64).cuda()
    k, v = qkv[:, 8:10], qkv[:, 10:]
    plan = eba.Rope((32,))
    a, b = p.on_gpu(eba), q.on_gpu(eba)
    eba.cache_append(a, k.contiguous(), v.contiguous(), p.gtable, p.glens, rope=plan)
    eba.cache_append(b, k, v, q.gtable, q.glens, rope=plan)
    assert torch.equal(p.gk.view(torch.uint8), q.gk.view(torch.uint8))
    assert torch.equal(p.gv.view(torch.uint8), q.gv.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eba.cache_append(b, k, v, q.gtable, q.glens, rope=plan)
    p.glens.sub_(1)
    q.glens.sub_(1)
    graph.replay()
    eba.cache_append(a, k, v, p.gtable, p.glens, rope=plan)
    assert torch.equal(p.gk.view(torch.uint8), q.gk.view(torch.uint8))


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("H,Hk,d,axes", [(8, 2, 128, (64,)), (4, 4, 64, (8, 12, 12))])
def test_prompt_then_tokens_through_the_cache(eba, H, Hk, d, axes):
    """Prompts rotated, attended to and appended; then tokens, one by one, appended
    and decoded: every token's output is the packed attention's over the same keys."""
    prompts, steps, page = [37, 100, 5], 4, 16
    B = len(prompts)
    g = torch.Generator().manual_seed(11)
    plan = eba.Rope(axes)
    total = [n + steps for n in prompts]
    per = [-(-n // page) for n in total]
    k_pages = torch.full((sum(per), page, Hk, d), math.nan, device="cuda", dtype=torch.bfloat16)
    v_pages = k_pages.clone()
    cache = eba.PagedCache(k_pages, v_pages)
    ids = torch.randperm(sum(per), generator=g).to(torch.int32)
    table = torch.full((B, max(per)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
    table = table.cuda()
    seqs = [(bf16(g, n, H, d), bf16(g, n, Hk, d), bf16(g, n, Hk, d),
             torch.randint(0, 500, (len(axes), n), generator=g).to(torch.int32)) for n in total]

    def rows(what, lo, hi):
        return torch.cat([s[what][lo(b):hi(b)] if what < 3 else s[3][:, lo(b):hi(b)]
                          for b, s in enumerate(seqs)], 0 if what < 3 else 1).cuda()

    lens = torch.tensor(prompts, dtype=torch.int32).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32)
    k, v, pos = (rows(w, lambda b: 0, lambda b: prompts[b]) for w in (1, 2, 3))
    eba.cache_append(cache, k, v, table, lens, cu.cuda(), rope=plan, positions=pos)
    for s in range(steps):
        lens += 1
        q, k, v, pos = (rows(w, lambda b: prompts[b] + s, lambda b: prompts[b] + s + 1) for w in range(4))
        eba.cache_append(cache, k, v, table, lens, rope=plan, positions=pos)
        o, lse = eba.decode(cache, q, table, lens, rope=plan, positions=pos)
        n = [p + s + 1 for p in prompts]
        cu_k = [0, *np.cumsum(n).tolist()]
        ka, va, pa = (rows(w, lambda b: 0, lambda b: n[b]) for w in (1, 2, 3))
        qr, _ = eba.rope_fwd(q, None, pos, plan)
        kr, _ = eba.rope_fwd(ka, None, pa, plan)
        o2, lse2 = eba.fwd_varlen(qr, kr, va, list(range(B + 1)), cu_k)
        # the same bf16 q, k, v: both are within the packed attention's bar of the exact result
        assert (o.float() - o2.float()).abs().max().item() <= 2e-2
        assert (lse - lse2.t()).abs().max().item() <= 1e-3
        ro, rl = oracle.varlen_forward(qr, kr, va, list(range(B + 1)), cu_k, 1 / math.sqrt(d))
        assert np.abs(np64(o) - ro).max() <= 2.0 ** -8 * np.abs(ro).max() + 1e-3
        assert np.abs(np64(lse) - rl.T).max() <= 1e-4


@pytest.mark.parametrize("longest", [100, 3000])
def test_calls_right_behind_each_other_see_what_was_written(eba, longest):
    """Rotate, append what was rotated, decode with it: 40 times over the same few
    addresses, with a pause after every call, without, and in a graph."""
    plan, pos = eba.Rope((64,)), torch.tensor([1, 77], device="cuda", dtype=torch.int32)
    start = bf16(torch.Generator().manual_seed(3), 2, 4, 128).cuda()
    p = Paged([longest, 64], 16, 2, 128, seed=9)
    cache = p.on_gpu(eba)

    def run(pause=lambda: None):
        x, outs = start, []
        for _ in range(40):
            x, _ = eba.rope_fwd(x, None, pos, plan)
            pause()
            eba.cache_append(cache, x[:, :2], x[:, 2:], p.gtable, p.glens)
            pause()
            outs.append(eba.decode(cache, x, p.gtable, p.glens)[0])
            pause()
        return torch.stack(outs)

    ref = run(torch.cuda.synchronize)
    assert torch.equal(run(), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        graph.replay()
        assert torch.equal(out, ref)
