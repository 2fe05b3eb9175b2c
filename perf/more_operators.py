"""Attention within a sliding window and to a few first tokens, attention of drafted tokens over the paged cache, and the
bookkeeping of the cache's pages: the cases that are measured, their plain forms in elementary torch operations, and
their definitions in 64 bits.

A case's "op" is one of
  window   q, k, v [B, H, L, d] -> o and the gradients of q, k, v; query i stands at key i + Lk - Lq and sees the keys from
           `left` before to `right` behind its place (-1: any number) and, up to `right` behind it, the first `sinks`
  decode   one new token per sequence over the last `window` and the first `sinks` of its cached keys; the pages between
           are not there
  tree     drafted tokens, the last ones of their sequences: each sees its context (within a window, and the sinks) and
           those drafted tokens that its mask names, or without a mask those before it
  step     a step of speculative decoding: append the drafted tokens, attend, move the accepted ones together
  pages    the page tables' turn: give pages back, let sequences fork, reserve room for new tokens, copy the pages that
           forked sequences do not share
  gather   chosen tokens of long sequences into pages of their own
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a short clip's local attention in a training step: latency
        dict(name="window_clip", op="window", B=2, H=4, Hkv=4, Lq=333, Lk=333, d=64, left=48, right=48, sinks=0),
        # training on long videos (64 x 14 x 14 tubelets): each token sees 8 frames back and the first frame's first tokens
        dict(name="window_causal", op="window", B=1, H=16, Hkv=4, Lq=12544, Lk=12544, d=128, left=1567, right=0, sinks=16),
        # 32 frames of 14 x 14, four frames to both sides and one class token that all see
        dict(name="window_video", op="window", B=2, H=16, Hkv=16, Lq=6273, Lk=6273, d=64, left=784, right=784, sinks=1),
        # one user far into a stream, whose layer keeps 1024 keys: latency
        dict(name="decode_window_one", op="decode", B=1, longest=20011, window=1024, sinks=4, H=32, Hkv=8, d=128, page=16, cache="bf16"),
        # a served batch of streams, a window of 4096
        dict(name="decode_window_batch", op="decode", B=64, longest=50021, window=4096, sinks=4, H=32, Hkv=8, d=128, page=32, cache="bf16"),
        # one user, a small tree: latency
        dict(name="tree_one", op="tree", B=1, longest=1501, new=16, masked=True, window=0, sinks=0, H=32, Hkv=8, d=128, page=16, cache="bf16"),
        # a served batch of very different lengths, trees of up to 32 tokens
        dict(name="tree_batch", op="tree", B=32, longest=8191, new=32, masked=True, window=0, sinks=0, H=32, Hkv=8, d=128, page=32, cache="bf16"),
        # very long e4m3 caches, drafted chains, eight heads on each key head
        dict(name="chain_long_e4m3", op="tree", B=8, longest=131071, new=12, masked=False, window=0, sinks=0, H=32, Hkv=4, d=128, page=128, cache="e4m3"),
        # the three calls of one layer in a step of speculative decoding, 16 heads of 64, pages that are no power of two
        dict(name="draft_step", op="step", B=16, longest=6007, new=24, masked=True, window=0, sinks=0, H=16, Hkv=16, d=64, page=48, cache="bf16"),
        # a beam search's turn: 64 slots, 24 of them taken by forks
        dict(name="pages_beams", op="pages", B=64, longest=2011, forks=24, grow=5, Hkv=8, d=128, page=16, cache="bf16", copy=True),
        # the bookkeeping of a server's whole card: half a million pages
        dict(name="pages_server", op="pages", B=512, longest=12544, forks=100, grow=64, Hkv=1, d=64, page=8, cache="bf16", copy=False),
        # heavy hitters of long caches are kept, the others go
        dict(name="gather_kept", op="gather", B=16, longest=12544, keep=2048, Hkv=8, d=128, page=16, cache="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "decode", "tree", "tree", "step", "pages", "gather"])
    d = rng.choice([64, 128])
    if op == "window":
        hkv, b = rng.choice([1, 2, 3, 4, 8, 16]), rng.randint(1, 4)
        h = hkv * rng.choice([1, 1, 2, 4, 5])
        most = int(math.sqrt(1_500_000_000 / (b * h)))
        lk = _log_int(rng, 1, min(12544, most))
        lq = rng.choice([lk, lk, _log_int(rng, 1, min(12544, most))])
        return dict(op=op, B=b, H=h, Hkv=hkv, Lq=lq, Lk=lk, d=d, left=rng.choice([-1, _log_int(rng, 1, lk), _log_int(rng, 1, lk)]),
                    right=rng.choice([0, 0, -1, _log_int(rng, 1, lk)]), sinks=rng.choice([0, 1, 4, _log_int(rng, 1, 300)]))
    hkv, b = rng.choice([1, 2, 3, 4, 8, 16]), _log_int(rng, 1, 64)
    c = dict(op=op, B=b, Hkv=hkv, d=d, page=rng.choice([8, 16, 20, 32, 48, 64, 128]), cache=rng.choice(["bf16", "bf16", "e4m3"]))
    if op == "pages":
        pages = 500_000 // b
        return c | dict(longest=_log_int(rng, 1, min(12544, pages * c["page"], 100_000_000 // (b * hkv * d))), forks=rng.randint(0, b // 2),
                        grow=_log_int(rng, 1, 100), copy=rng.choice([True, False]))
    if op == "gather":
        n = _log_int(rng, 1, min(30000, 200_000_000 // (b * hkv * d)))
        return c | dict(longest=n, keep=_log_int(rng, 1, n))
    c |= dict(H=hkv * rng.choice([1, 2, 4, 5, 8, 16]), sinks=rng.choice([0, 1, 4, _log_int(rng, 1, 200)]))
    if op == "decode":
        most = 200_000_000 // (b * hkv * d)
        return c | dict(longest=_log_int(rng, 1, 60000), window=_log_int(rng, 1, min(8192, most)))
    c |= dict(new=_log_int(rng, 1, 64), masked=rng.choice([True, False]))
    most = min(130000, 200_000_000 // (b * hkv * d), 4_000_000_000 // (b * c["H"] * c["new"]))
    n = _log_int(rng, c["new"], max(c["new"], most))
    return c | dict(longest=n, window=rng.choice([0, 0, _log_int(rng, 1, n)]))


def _lens(case):
    """How many keys each sequence holds: the longest one, and others spread evenly below it."""
    b, longest = case["B"], case["longest"]
    low = max(case.get("new", 1), longest // 8)
    r = random.Random(b * 1000003 + longest)
    return [longest] + [r.randint(low, longest) for _ in range(b - 1)]


def _news(case):
    """Drafted tokens of each sequence: the most in the first."""
    r = random.Random(case["B"] * 7919 + case["new"])
    return [case["new"]] + [r.randint(max(1, case["new"] // 2), case["new"]) for _ in range(case["B"] - 1)]


def _kept(case):
    """Tokens that each sequence keeps."""
    r = random.Random(case["B"] * 104729 + case["keep"])
    return [min(n, r.randint(max(1, case["keep"] // 2), case["keep"])) for n in _lens(case)]


def _scales(case):
    return (0.0125, 0.011) if case["cache"] == "e4m3" else (1.0, 1.0)


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _trees(case, rng):
    """Each drafted token's ancestors and itself, one bit a token; it hangs on one of the last few before it, or on none. And
    the places of one path from a root, as a verification accepts it."""
    masks, paths = [], []
    for n in _news(case):
        mine, line = [], []
        for i in range(n):
            p = i - 1 if not case["masked"] else rng.randint(max(-1, i - 6), i - 1)
            mine.append((mine[p] if p >= 0 else 0) | 1 << i)
            line.append((line[p] if p >= 0 else []) + [i])
        masks += [m - (1 << 64) if m >> 63 else m for m in mine]
        paths.append(line[rng.randrange(n)])
    return masks, paths


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    dev = torch.device("cuda")

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    def ints(x):
        return torch.tensor(x, device=dev, dtype=torch.int32)

    op, d, hkv = case["op"], case["d"], case["Hkv"]
    s = dict(case=case)
    if op == "window":
        b, h = case["B"], case["H"]
        s["q"] = normal(b, h, case["Lq"], d).requires_grad_(True)
        s["k"] = normal(b, hkv, case["Lk"], d).requires_grad_(True)
        s["v"] = normal(b, hkv, case["Lk"], d).requires_grad_(True)
        s["g"] = normal(b, h, case["Lq"], d)
    else:
        b, page, lens = case["B"], case["page"], _lens(case)
        s["lens"] = ints(lens)
        first = [0] * b  # the first page of a sequence behind its sinks that is still there
        if op == "decode":
            first = [max(0, n - case["window"]) // page for n in lens]
        sunk = [-(-case.get("sinks", 0) // page)] * b
        per = [-(-n // page) for n in lens]
        room = [-(-case["grow"] // page) + 1 if op == "pages" else 0] * b
        here = [[e for e in range(n) if e >= f or e < u] for n, f, u in zip(per, first, sunk)]
        used, wide = sum(map(len, here)), max(x + r for x, r in zip(per, room))
        to = [-(-n // page) for n in _kept(case)] if op == "gather" else []
        pages = used + sum(to) + sum(room) + (case["forks"] if op == "pages" else 0) + 7
        order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
        flat = torch.full((b * wide,), -1, device=dev, dtype=torch.int32)  # -1: no page
        flat[torch.tensor([i * wide + e for i, x in enumerate(here) for e in x], device=dev)] = order[:used]
        s["table"] = flat.view(b, wide)
        if op != "pages" or case["copy"]:
            ks, vs = _scales(case)
            s["kc"], s["vc"] = normal(pages, page, hkv, d), normal(pages, page, hkv, d)
            if case["cache"] == "e4m3":
                s["kc"] = (s["kc"].float() / ks).clamp(-448, 448).to(E4M3)
                s["vc"] = (s["vc"].float() / vs).clamp(-448, 448).to(E4M3)
        if op == "decode":
            s["q"] = normal(b, case["H"], d)
        if op in ("tree", "step"):
            news = _news(case)
            t = sum(news)
            s["q"], s["cu"] = normal(t, case["H"], d), ints(_starts(news))
            masks, paths = _trees(case, rng)
            s["mask"] = torch.tensor(masks, device=dev, dtype=torch.int64) if case["masked"] else None
            if op == "step":
                s["k"], s["v"] = normal(t, hkv, d), normal(t, hkv, d)
                # what a verification accepted: the places of one path's tokens, and how many of each sequence
                before = [n - m for n, m in zip(lens, news)]
                s["before"], s["cu_kept"] = ints(before), ints(_starts([len(p) for p in paths]))
                s["places"] = ints([f + i for f, p in zip(before, paths) for i in p])
        if op == "pages":
            s["refs"] = torch.zeros(pages, device=dev, dtype=torch.int32)
            s["refs"][order[:used].long()] = 1
            slots = rng.sample(range(b), b)
            into, left = slots[:case["forks"]], slots[case["forks"]:]
            s["src"], s["dst"] = ints([rng.choice(left) for _ in into]), ints(into)
            s["from"] = torch.zeros(b, device=dev, dtype=torch.int32)
            s["to"] = torch.zeros(b, device=dev, dtype=torch.int32)
            s["to"][s["dst"].long()] = wide * page  # the slots that forks take give back all that they hold
        if op == "gather":
            kept = _kept(case)
            s["places"] = torch.cat([torch.randperm(n, generator=g, device=dev)[:m].sort().values for n, m in zip(lens, kept)]).to(torch.int32)
            s["cu"] = ints(_starts(kept))
            new = torch.full((b * max(to),), -1, device=dev, dtype=torch.int32)
            new[torch.tensor([i * max(to) + e for i, n in enumerate(to) for e in range(n)], device=dev)] = order[used:used + sum(to)]
            s["new_table"] = new.view(b, max(to))
    if own:
        import exact_blockwise_attention_gb300 as eba

        s["eba"] = eba
        if "kc" in s:
            s["cache"] = eba.PagedCache(s["kc"], s["vc"], *_scales(case))
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------

def _window(s):
    case = s["case"]
    b, h, hkv, lq, lk, d = (case[n] for n in ("B", "H", "Hkv", "Lq", "Lk", "d"))
    c = 1 / math.sqrt(d)
    q, g = (s[n].detach().float().reshape(b, hkv, -1, d) for n in ("q", "g"))  # a key head's query heads, one behind the other
    k, v = s["k"].detach().float(), s["v"].detach().float()
    place = torch.arange(lq, device=q.device)[:, None] + (lk - lq)
    key = torch.arange(lk, device=q.device)[None]
    left = case["left"] if case["left"] >= 0 else lk + lq
    right = case["right"] if case["right"] >= 0 else lk + lq
    seen = (key <= place + right) & ((key >= place - left) | (key < case["sinks"]))
    seen = seen.repeat(h // hkv, 1)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(c).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total > 0, total, 1.0))
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(-1, -2), g)
    ds = torch.matmul(g, v.transpose(-1, -2)).sub_((g * o).sum(-1, keepdim=True)).mul_(p).mul_(c)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(-1, -2), q)
    return [y.to(torch.bfloat16) for y in (o.reshape(b, h, lq, d), dq.reshape(b, h, lq, d), dk, dv)]


def _attend(x, seen, v):
    """Softmax over the keys that are seen, times the values; a row that sees none is 0, its lse -inf."""
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0), (top + total.log())[..., 0]


def _cached(s, places, there):
    """Keys [b, heads, d, n] and values [b, heads, n, d] of a batch's places [b, n], 0 where there is none."""
    case = s["case"]
    ks, vs = _scales(case)
    places = torch.where(there, places, 0)
    page = torch.where(there, s["table"].gather(1, (places // case["page"]).clamp(max=s["table"].shape[1] - 1)), 0).long()
    slot = places % case["page"]
    k = s["kc"][page, slot].float() * ks
    v = torch.where(there[..., None, None], s["vc"][page, slot].float() * vs, 0.0)
    return k.permute(0, 2, 3, 1), v.permute(0, 2, 1, 3)


def _decode(s):
    case = s["case"]
    b, h, hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    n = s["lens"].long()[:, None]
    back = torch.arange(case["window"], device=n.device)[None]
    near = n - case["window"] + back
    sink = torch.arange(case["sinks"], device=n.device)[None].expand(b, -1)
    places = torch.cat([sink, near], 1)
    there = torch.cat([(sink < n) & (sink < n - case["window"]), near >= 0], 1)  # a sink within the window counts once
    k, v = _cached(s, places, there)
    x = torch.matmul(s["q"].float().reshape(b, hkv, h // hkv, d), k) / math.sqrt(d)
    o, lse = _attend(x, there[:, None, None], v)
    return o.reshape(b, h, d).to(torch.bfloat16), lse.reshape(b, h)


def _tree(s):
    case = s["case"]
    b, h, hkv, d, most = case["B"], case["H"], case["Hkv"], case["d"], case["new"]
    cu, lens, t = s["cu"].long(), s["lens"].long(), s["q"].shape[0]
    dev = cu.device
    row = torch.arange(t, device=dev)
    seq = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[seq]
    at = (cu[:-1, None] + torch.arange(most, device=dev)).clamp(max=t - 1)  # [b, most]: a sequence's rows, and others behind them
    new = (cu[1:] - cu[:-1])[:, None]
    before = lens[:, None] - new
    key = torch.arange(case["longest"], device=dev)[None].expand(b, -1)
    k, v = _cached(s, key, key < lens[:, None])
    draft = key - before  # a key's number among the drafted ones
    if case["masked"]:
        bits = s["mask"][at]
        among = (bits[:, :, None] >> draft.clamp(0, 63)[:, None]) & 1 > 0
        depth = ((bits[:, :, None] >> torch.arange(64, device=dev)) & 1).sum(-1) - 1
    else:
        depth = torch.arange(most, device=dev)[None].expand(b, -1)
        among = draft[:, None] <= depth[:, :, None]
    place = (before + depth)[:, :, None]
    near = torch.ones_like(among) if case["window"] == 0 else (key[:, None] > place - case["window"]) | (key[:, None] < case["sinks"])
    seen = torch.where((draft < 0)[:, None], near, among & (near if not case["masked"] else True)) & (key < lens[:, None])[:, None]
    q = s["q"][at].float().reshape(b, most, hkv, h // hkv, d).transpose(1, 2).reshape(b, hkv, -1, d)
    x = torch.matmul(q, k) / math.sqrt(d)
    o, lse = _attend(x, seen.repeat_interleave(h // hkv, 1)[:, None], v)
    o = o.reshape(b, hkv, most, h // hkv, d).transpose(1, 2).reshape(b, most, h, d)[seq, i]
    lse = lse.reshape(b, hkv, most, h // hkv).transpose(1, 2).reshape(b, most, h)[seq, i]
    return o.to(torch.bfloat16), lse


def _step(s):
    case = s["case"]
    ks, vs = _scales(case)
    size = case["page"]
    cu, t = s["cu"].long(), s["q"].shape[0]
    row = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    at = s["before"].long()[b] + row - cu[b]
    page, slot = s["table"][b, at // size].long(), at % size
    if case["cache"] == "e4m3":
        s["kc"][page, slot] = (s["k"].float() / ks).clamp(-448, 448).to(E4M3)
        s["vc"][page, slot] = (s["v"].float() / vs).clamp(-448, 448).to(E4M3)
    else:
        s["kc"][page, slot], s["vc"][page, slot] = s["k"], s["v"]
    o, lse = _tree(s)
    _move(s, s["table"], s["cu_kept"].long(), s["before"].long())
    return o, lse, s["kc"], s["vc"]


def _move(s, new_table, cu, start):
    size = s["case"]["page"]
    row = torch.arange(s["places"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    old, at = s["places"].long(), start[b] + row - cu[b]
    page, slot = s["table"][b, old // size].long(), old % size
    to, where = new_table[b, at // size].long(), at % size
    for c in (s["kc"], s["vc"]):
        c = c.view(torch.int16 if c.dtype == torch.bfloat16 else torch.int8)
        c[to, where] = c[page, slot]


def _give(refs, want):
    """The lowest free pages, one for each that is wanted, in order; -1 where none is left. Counts them in `refs`."""
    free = refs == 0
    rank = free.cumsum(0) - 1
    n = refs.shape[0]
    order = torch.full((n + 1,), -1, device=refs.device, dtype=torch.int32)
    order[torch.where(free, rank, n)] = torch.where(free, torch.arange(n, device=refs.device, dtype=torch.int32), -1)
    order[n] = -1
    nth = (want.flatten().cumsum(0) - 1).clamp(min=0, max=n).view(want.shape)
    got = torch.where(want, order[nth], -1)
    refs.scatter_add_(0, got.clamp(min=0).flatten().long(), (got >= 0).flatten().int())
    return got


def _pages(s):
    size = s["case"]["page"]
    table, refs, lens = s["table"].clone(), s["refs"].clone(), s["lens"].clone()
    entry = torch.arange(table.shape[1], device=table.device)[None]
    # give back the pages that lie wholly within [from, to)
    gone = (entry >= (s["from"] + size - 1)[:, None] // size) & (entry < s["to"][:, None] // size) & (table >= 0)
    refs.scatter_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().int())
    table = torch.where(gone, -1, table)
    # fork: whole pages are shared, the last one is copied where it is not full
    src, dst = s["src"].long(), s["dst"].long()
    n, rows = lens[src][:, None], table[src]
    shared, partly = (entry < n // size) & (rows >= 0), (entry == n // size) & (n % size > 0) & (rows >= 0)
    refs.scatter_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().int())
    some = partly.any(1)
    new = _give(refs, some)
    old = torch.where(some & (new >= 0), torch.where(partly, rows, 0).sum(1), -1).int()
    table[dst] = torch.where(shared, rows, torch.where(partly, new[:, None], -1))
    lens[dst] = lens[src]
    # reserve
    more = lens + s["case"]["grow"]
    want = (entry >= ((lens + size - 1) // size)[:, None]) & (entry < ((more + size - 1) // size)[:, None]) & (table < 0)
    table = torch.where(want, _give(refs, want), table)
    out = [table, refs, lens, old, new]
    if s["case"]["copy"]:
        at, to = old.long(), new.long()
        at, to = torch.where(to >= 0, at, 0), torch.where(to >= 0, to, 0)  # nothing to copy: page 0 onto itself
        for c in (s["kc"], s["vc"]):
            c = c.view(torch.int16 if c.dtype == torch.bfloat16 else torch.int8)
            c[to] = c[at]
        out += [s["kc"], s["vc"]]
    return out


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "window":
        return _window(s)
    if op == "decode":
        return _decode(s)
    if op == "tree":
        return _tree(s)
    if op == "step":
        return _step(s)
    if op == "pages":
        return _pages(s)
    _move(s, s["new_table"], s["cu"].long(), torch.zeros_like(s["lens"]).long())
    return s["kc"], s["vc"]


# ---- the framework's calls -------------------------------------------------------------------------------------------

def _own(s):
    eba, case = s["eba"], s["case"]
    op = case["op"]
    if op == "window":
        left, right = (None if case[n] < 0 else case[n] for n in ("left", "right"))
        o = eba.attention_window(s["q"], s["k"], s["v"], left, right, case["sinks"])
        return [o, *torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["g"])]
    if op == "decode":
        return eba.decode(s["cache"], s["q"], s["table"], s["lens"], window=case["window"], sinks=case["sinks"])
    if op in ("tree", "step"):
        if op == "step":
            eba.cache_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["cu"])
        o, lse = eba.decode_tree(s["cache"], s["q"], s["table"], s["lens"], s["cu"], mask=s["mask"], window=case["window"] or None,
                                 sinks=case["sinks"])
        if op == "tree":
            return o, lse
        eba.cache_gather(s["cache"], s["table"], s["places"], s["cu_kept"], to_start=s["before"])
        return o, lse, s["kc"], s["vc"]
    if op == "gather":
        eba.cache_gather(s["cache"], s["table"], s["places"], s["cu"], to_table=s["new_table"])
        return s["kc"], s["vc"]
    table, refs, lens = s["table"].clone(), s["refs"].clone(), s["lens"].clone()
    pool = eba.PagePool(refs, case["page"])
    eba.pages_release(pool, table, s["from"], s["to"])
    old, new = eba.pages_fork(pool, table, lens, s["src"], s["dst"])
    eba.pages_reserve(pool, table, lens, lens + case["grow"])
    out = [table, refs, lens, old, new]
    if case["copy"]:
        eba.cache_copy(s["cache"], old, new)
        out += [s["kc"], s["vc"]]
    return out


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def _pairs(case):
    """How many (query, key) pairs of one head are seen."""
    lq, lk, left, right, sinks = (case[n] for n in ("Lq", "Lk", "left", "right", "sinks"))
    total = 0
    for i in range(lq):
        place = i + lk - lq
        hi = min(lk, place + right + 1) if right >= 0 else lk
        lo = max(0, place - left) if left >= 0 else 0
        total += max(0, hi - lo) + max(0, min(sinks, hi, lo))
    return total


def work(case):
    op, d, hkv, b = case["op"], case["d"], case["Hkv"], case["B"]
    size = 1 if case.get("cache") == "e4m3" else 2
    if op == "window":
        q, k = b * case["H"] * case["Lq"] * d, b * hkv * case["Lk"] * d
        return {"bytes": 2 * (4 * q + 4 * k), "flops": 14 * d * b * case["H"] * _pairs(case)}
    lens, page = _lens(case), case["page"]
    row = hkv * d * 2 * size  # a token's keys and values
    if op == "decode":
        n = sum(min(x, case["window"]) + min(case["sinks"], max(0, x - case["window"])) for x in lens)
        return {"bytes": n * row + b * case["H"] * (d * 4 + 4) + 4 * n // page, "flops": 4 * n * case["H"] * d}
    if op in ("tree", "step"):
        news = _news(case)
        near = [n if case["window"] == 0 else min(n, case["window"] + m + case["sinks"]) for n, m in zip(lens, news)]
        t = sum(news)
        nbytes = sum(near) * row + t * case["H"] * (d * 4 + 4) + 4 * sum(near) // page + (8 * t if case["masked"] else 0)
        if op == "step":  # append the drafted tokens; move about half of the accepted ones, some eighth of all
            nbytes += t * hkv * d * 2 * (2 + size) + t // 8 * row * 2
        return {"bytes": nbytes, "flops": 4 * d * case["H"] * sum(n * m for n, m in zip(near, news))}
    if op == "gather":
        return {"bytes": sum(_kept(case)) * (2 * row + 4), "flops": 0}
    entries = sum(-(-n // page) for n in lens)
    copied = case["forks"] * page * row * 2 if case["copy"] else 0
    return {"bytes": 4 * 2 * 2 * entries + copied, "flops": 0}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def _exact_window(case, s):
    """Head by head, the gradients by automatic differentiation."""
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=s[n].device) for n in ("q", "k", "v")}
    o = torch.zeros_like(out["q"])
    lq, lk = case["Lq"], case["Lk"]
    i = torch.arange(lq, device=o.device)[:, None]
    j = torch.arange(lk, device=o.device)[None, :] - (lk - lq)  # the query that stands at the key
    hidden = torch.zeros(lq, lk, dtype=torch.bool, device=o.device)
    if case["left"] >= 0:
        hidden |= (i - j > case["left"]) & (j + (lk - lq) >= case["sinks"])
    if case["right"] >= 0:
        hidden |= j - i > case["right"]
    blind = hidden.all(1)
    for b in range(case["B"]):
        for h in range(case["H"]):
            kh = h // (case["H"] // case["Hkv"])
            q, k, v = (x.detach().double().requires_grad_(True) for x in (s["q"][b, h], s["k"][b, kh], s["v"][b, kh]))
            x = (q @ k.t() / math.sqrt(case["d"])).masked_fill(hidden, -math.inf).masked_fill(blind[:, None], 0.0)
            y = (torch.softmax(x, -1) @ v) * (~blind[:, None])
            gq, gk, gv = torch.autograd.grad(y, (q, k, v), s["g"][b, h].double())
            o[b, h], out["q"][b, h] = y.detach(), gq
            out["k"][b, kh] += gk
            out["v"][b, kh] += gv
    return [o, out["q"], out["k"], out["v"]]


def _exact_rows(case, s, b, q, seen):
    """Attention of q [t, H, d] over the keys of sequence b that are seen [t, n] (those that no row sees need not be there)."""
    ks, vs = _scales(case)
    used = seen.any(0).nonzero()[:, 0]
    page, slot = s["table"][b].long()[used // case["page"]], used % case["page"]
    k, v = ks * s["kc"][page, slot].double(), vs * s["vc"][page, slot].double()
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for h in range(case["H"] if used.numel() else 0):
        g = h // (case["H"] // case["Hkv"])
        x = (q[:, h].double() @ k[:, g].t() / math.sqrt(case["d"])).masked_fill(~seen[:, used], -math.inf)
        lse[:, h] = torch.logsumexp(x, -1)
        o[:, h] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v[:, g]
    return o, lse


def _exact_tree(case, s):
    out = []
    news, lens = _news(case), _lens(case)
    masks = s["mask"].tolist() if case["masked"] else None
    at = 0
    for b, (m, n) in enumerate(zip(news, lens)):
        key = torch.arange(n, device=s["q"].device)
        seen = []
        for i in range(m):
            bits = [masks[at + i] >> j & 1 for j in range(m)] if case["masked"] else [int(j <= i) for j in range(m)]
            place = n - m + sum(bits) - 1
            near = (key > place - case["window"]) | (key < case["sinks"]) if case["window"] else key >= 0
            drafted = torch.zeros(n, dtype=torch.bool, device=key.device)
            drafted[n - m:] = torch.tensor(bits, device=key.device) > 0
            seen.append(torch.where(key < n - m, near, drafted if case["masked"] else drafted & near))
        out.append(_exact_rows(case, s, b, s["q"][at:at + m], torch.stack(seen)))
        at += m
    return [torch.cat([x[i] for x in out]) for i in (0, 1)]


def _exact_pages(case, s):
    size, table, refs, lens = case["page"], s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    for b, (x, y) in enumerate(zip(s["from"].tolist(), s["to"].tolist())):
        for e in range(len(table[b])):
            if x <= e * size and (e + 1) * size <= y and table[b][e] >= 0:
                refs[table[b][e]] -= 1
                table[b][e] = -1
    old, new, free = [], [], 0

    def give():
        nonlocal free
        while free < len(refs) and refs[free]:
            free += 1
        if free == len(refs):
            return -1
        refs[free] = 1
        return free

    pairs = list(zip(s["src"].tolist(), s["dst"].tolist()))
    for a, b in pairs:
        for e in range(lens[a] // size):
            if table[a][e] >= 0:
                refs[table[a][e]] += 1
    for a, b in pairs:
        whole = lens[a] // size
        table[b] = table[a][:whole] + [-1] * (len(table[a]) - whole)
        lens[b] = lens[a]
        part = table[a][whole] if lens[a] % size else -1
        new.append(give() if part >= 0 else -1)
        old.append(part if new[-1] >= 0 else -1)
        if part >= 0:
            table[b][whole] = new[-1]
    for b, n in enumerate(lens):
        for e in range(-(-n // size), -(-(n + case["grow"]) // size)):
            if table[b][e] < 0:
                table[b][e] = give()
    out = [torch.tensor(x, dtype=torch.int32) for x in (table, refs, lens, old, new)]
    if case["copy"]:
        for c in (s["kc"], s["vc"]):
            c = c.double()
            for x, y in zip(old, new):
                if y >= 0:
                    c[y] = c[x]
            out.append(c)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "window":
        return _exact_window(case, s)
    if op == "pages":
        return _exact_pages(case, s)
    lens, size = _lens(case), case["page"]
    if op == "decode":
        out = []
        for b, n in enumerate(lens):
            key = torch.arange(n, device=s["q"].device)
            seen = (key >= n - case["window"]) | (key < case["sinks"])
            out.append(_exact_rows(case, s, b, s["q"][b:b + 1], seen[None]))
        return [torch.cat([x[i] for x in out]) for i in (0, 1)]
    table = s["table"].tolist()
    if op == "step":  # the attention reads what the cache holds
        ks, vs = _scales(case)
        for c, x, f in ((s["kc"], s["k"], ks), (s["vc"], s["v"], vs)):
            x = x.double() / f if case["cache"] == "bf16" else (x.double() / f).clamp(-448, 448)
            at = _starts(_news(case))
            for b, n in enumerate(lens):
                for i in range(at[b], at[b + 1]):
                    p = n - at[b + 1] + i
                    c[table[b][p // size], p % size] = x[i].to(c.dtype)
    if op == "tree" or op == "step":
        out = _exact_tree(case, s)
        if op == "tree":
            return out
    kc, vc = s["kc"].double(), s["vc"].double()
    places, cu = s["places"].tolist(), s["cu_kept" if op == "step" else "cu"].tolist()
    to = table if op == "step" else s["new_table"].tolist()
    for b in range(case["B"]):
        mine = places[cu[b]:cu[b + 1]]
        start = s["before"].tolist()[b] if op == "step" else 0
        at = [start + i for i in range(len(mine))]
        a = [table[b][p // size] for p in mine], [p % size for p in mine]
        z = [to[b][p // size] for p in at], [p % size for p in at]
        for c in (kc, vc):
            c[z] = c[a].clone()
    return [*out, kc, vc] if op == "step" else [kc, vc]
