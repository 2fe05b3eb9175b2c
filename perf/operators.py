"""The position rotation, the paged key-value cache and the attention of one new token over it: the cases that are
measured, their plain forms in elementary torch operations, and their definitions in 64 bits.

A case's "op" is one of
  rope        q, k -> rotated q, k, laid out [B, H, L, d] or token-major [T, H, d]
  rope_train  the same with the gradients of q and k
  append      new keys (rotated) and values into the pages of a cache, bf16 or e4m3
  decode      one new token per sequence over its cached keys and values
  step        a serving step: append one token per sequence, then decode with the query rotated on the way (and held in
              bf16, as rope gives it)
"""
import math
import random

import torch

own = False

THETA = 10000.0
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # the new tokens of a small batch while it is served: q and k of 8 tokens, where latency counts
        dict(name="rope_tokens", op="rope", layout="thd", B=1, L=8, H=32, Hkv=8, d=128, axes="64", pairing="half", far=4000000),
        # the batch of the ViT-L video workload, 16 clips of 8 x 14 x 14 tubelets, one grid of positions for all clips
        dict(name="rope_clips", op="rope", layout="bhld", B=16, L=1568, H=16, Hkv=16, d=64, axes="8,12,12", pairing="half", far=14),
        # a training step's rotation of packed images and videos, grouped heads, neighbouring elements as pairs
        dict(name="rope_train_packed", op="rope_train", layout="thd", B=1, L=25088, H=16, Hkv=4, d=128, axes="20,22,22", pairing="interleaved", far=128),
        # one token per sequence of a batch that is served
        dict(name="append_tokens", op="append", B=32, new=1, longest=4000, Hkv=8, d=128, page=16, cache="bf16", axes="20,22,22", pairing="half"),
        # long prompts of several users at once into an e4m3 cache
        dict(name="append_prompts_e4m3", op="append", B=5, new=4999, longest=9000, Hkv=8, d=128, page=16, cache="e4m3", axes="64", pairing="half"),
        # a 128-frame video (64 x 14 x 14 tubelets) of 16 heads of 64
        dict(name="append_video", op="append", B=2, new=12544, longest=12600, Hkv=16, d=64, page=48, cache="bf16", axes="8,12,12", pairing="half"),
        # one user, a short cache: latency
        dict(name="decode_one_short", op="decode", B=1, longest=333, H=32, Hkv=8, d=128, page=16, cache="bf16", empty=0),
        # a served batch of very different lengths, grouped heads, with slots that hold no sequence
        dict(name="decode_batch_ragged", op="decode", B=64, longest=8191, H=32, Hkv=8, d=128, page=16, cache="bf16", empty=3),
        # the long-visual workload's keys (36864 of 32 heads of 128), one query token
        dict(name="decode_long_visual", op="decode", B=2, longest=36864, H=32, Hkv=32, d=128, page=64, cache="bf16", empty=0),
        # very long e4m3 caches, sixteen query heads on each key head
        dict(name="decode_long_e4m3", op="decode", B=8, longest=131071, H=64, Hkv=4, d=128, page=128, cache="e4m3", empty=0),
        # long videos (12544 tokens) of 16 heads of 64, pages that are no power of two
        dict(name="decode_videos_d64", op="decode", B=16, longest=12544, H=16, Hkv=16, d=64, page=48, cache="bf16", empty=0),
        # the two calls of a serving step of one layer
        dict(name="serving_step", op="step", B=48, longest=6007, H=32, Hkv=8, d=128, page=32, cache="bf16", empty=0, axes="20,22,22", pairing="half"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_axes(rng, d):
    pairs = rng.choice([d // 2, d // 2, d // 4])  # the whole head, or its first half
    n = rng.choice([1, 2, 3])
    cuts = sorted(rng.sample(range(1, pairs), n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))


def draw(rng):
    op = rng.choice(["rope", "rope_train", "append", "decode", "decode", "step"])
    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8, 16])
    c = dict(op=op, d=d, Hkv=hkv)
    if op in ("rope", "rope_train"):
        layout = rng.choice(["thd", "bhld"])
        b = 1 if layout == "thd" else rng.randint(1, 16)
        most = 60_000_000 // (hkv * 4 * d * b)
        c |= dict(layout=layout, B=b, L=_log_int(rng, 1, min(30000, most)), H=hkv * rng.choice([1, 2, 4]), far=_log_int(rng, 8, 4000000))
    else:
        c |= dict(page=rng.choice([8, 16, 20, 32, 48, 64, 128]), cache=rng.choice(["bf16", "bf16", "e4m3"]))
        b = _log_int(rng, 1, 64)
        if op == "append":
            new = rng.choice([1, _log_int(rng, 1, max(1, 50_000_000 // (b * hkv * d * 2)))])
            new = min(new, 20000)
            c |= dict(B=b, new=new, longest=new + rng.randint(0, 2000))
        else:
            most = 400_000_000 // (b * hkv * d * 2)
            c |= dict(B=b, longest=_log_int(rng, 1 + (op == "step"), min(130000, most)), H=hkv * rng.choice([1, 2, 4, 5, 8, 16]), empty=rng.choice([0, 0, 1]) if op == "decode" and b > 1 else 0)
    if op != "decode":
        c |= dict(axes=_draw_axes(rng, d), pairing=rng.choice(["half", "interleaved"]))
    return c


def _axes(case):
    return [int(x) for x in case["axes"].split(",")]


def _frequencies(case):
    """Each pair's frequency (radians a position) and axis: axis a's n pairs run through theta^(-i/n)."""
    f, a = [], []
    for i, n in enumerate(_axes(case)):
        f += [THETA ** (-j / n) for j in range(n)]
        a += [i] * n
    return f, a


def _lens(case):
    """How many keys each sequence holds: the longest one, and others spread evenly below it; the last `empty` hold none."""
    b, longest = case["B"], case["longest"]
    new = case.get("new", 1 if case["op"] == "step" else 0)
    low = max(new, 1, longest // 8)
    r = random.Random(b * 1000003 + longest)
    n = [longest] + [r.randint(low, longest) for _ in range(b - 1)]
    for i in range(case.get("empty", 0)):
        n[b - 1 - i] = 0
    return n


def _scales(case):
    return (0.0125, 0.011) if case["cache"] == "e4m3" else (1.0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    op, d, hkv = case["op"], case["d"], case["Hkv"]
    s = dict(case=case)
    if "axes" in case:
        f, a = _frequencies(case)
        s["freq"] = torch.tensor(f, device=dev, dtype=torch.float64)
        s["axis"] = torch.tensor(a, device=dev)
    if op in ("rope", "rope_train"):
        b, n, h = case["B"], case["L"], case["H"]
        shape = (lambda x: (n, x, d)) if case["layout"] == "thd" else (lambda x: (b, x, n, d))
        s["q"], s["k"] = normal(*shape(h)), normal(*shape(hkv))
        s["pos"] = torch.randint(0, case["far"], (len(_axes(case)), n), generator=g, device=dev, dtype=torch.int32)
        if op == "rope_train":
            s["gq"], s["gk"] = normal(*shape(h)), normal(*shape(hkv))
            s["q"].requires_grad_(True)
            s["k"].requires_grad_(True)
    else:
        b, page, lens = case["B"], case["page"], _lens(case)
        per = [-(-n // page) for n in lens]
        used, wide = sum(per), max(per)
        pages = used + 7
        kc, vc = normal(pages, page, hkv, d), normal(pages, page, hkv, d)
        ks, vs = _scales(case)
        if case["cache"] == "e4m3":
            kc = (kc.float() / ks).clamp(-448, 448).to(E4M3)
            vc = (vc.float() / vs).clamp(-448, 448).to(E4M3)
        order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)[:used]
        table = torch.full((b, wide), -1, device=dev, dtype=torch.int32)  # -1: no page
        has = torch.arange(wide, device=dev)[None] < torch.tensor(per, device=dev)[:, None]
        table[has] = order
        s |= dict(kc=kc, vc=vc, table=table, lens=torch.tensor(lens, device=dev, dtype=torch.int32))
        if op in ("append", "step"):
            new = case.get("new", 1)
            t = b * new
            s["k"], s["v"] = normal(t, hkv, d), normal(t, hkv, d)
            s["pos"] = torch.randint(0, 2 * case["longest"], (len(_axes(case)), t), generator=g, device=dev, dtype=torch.int32)
            s["cu"] = None if new == 1 else torch.arange(b + 1, device=dev, dtype=torch.int32) * new
        if op in ("decode", "step"):
            s["q"] = normal(b, case["H"], d)
    if own:
        import exact_blockwise_attention_gb300 as eba

        s["eba"] = eba
        if "axes" in case:
            s["plan"] = eba.Rope(_axes(case), theta=THETA, pairing=case["pairing"])
        if "kc" in s:
            s["cache"] = eba.PagedCache(s["kc"], s["vc"], *_scales(case))
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------

def _turn(s, x, sign=1.0):
    """x [..., tokens, heads, d] rotated by its tokens' angles: angles in 64 bits, the rotation in 32."""
    at = s["pos"].double()[s["axis"]].t() * s["freq"]  # [tokens, pairs]
    c, n = at.cos().float()[:, None], (sign * at.sin()).float()[:, None]
    r = s["freq"].numel()
    x = x.float()
    rot, rest = x[..., : 2 * r], x[..., 2 * r:]
    if s["case"]["pairing"] == "half":
        a, b = rot[..., :r], rot[..., r:]
        return torch.cat([a * c - b * n, a * n + b * c, rest], -1)
    a, b = rot[..., 0::2], rot[..., 1::2]
    return torch.cat([torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2), rest], -1)


def _rope(s, x, sign=1.0):
    x = x.detach()
    if s["case"]["layout"] == "thd":
        return _turn(s, x, sign).to(torch.bfloat16)
    return _turn(s, x.transpose(1, 2), sign).transpose(1, 2).to(torch.bfloat16).contiguous()


def _append(s):
    case = s["case"]
    t = torch.arange(s["k"].shape[0], device=s["k"].device)
    new = case.get("new", 1)
    b = t // new
    at = s["lens"][b].long() - (new - t % new)
    page, slot = s["table"][b, at // case["page"]].long(), at % case["page"]
    k, v = _turn(s, s["k"]), s["v"].float()
    if case["cache"] == "e4m3":
        ks, vs = _scales(case)
        s["kc"][page, slot] = (k / ks).clamp(-448, 448).to(E4M3)
        s["vc"][page, slot] = (v / vs).clamp(-448, 448).to(E4M3)
    else:
        s["kc"][page, slot] = k.to(torch.bfloat16)
        s["vc"][page, slot] = s["v"]


def _decode(s, q):
    case = s["case"]
    b, h, hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    ks, vs = _scales(case)
    at = s["table"].clamp(min=0).long()
    n = at.shape[1] * case["page"]
    k = s["kc"][at].reshape(b, n, hkv, d).permute(0, 2, 3, 1).float() * ks
    v = s["vc"][at].reshape(b, n, hkv, d).permute(0, 2, 1, 3).float() * vs
    held = torch.arange(n, device=q.device)[None] < s["lens"][:, None]
    x = torch.matmul(q.float().reshape(b, hkv, h // hkv, d), k) / math.sqrt(d)
    x = torch.where(held[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(held[:, None, :, None], v, 0.0)) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).reshape(b, h)
    return o.reshape(b, h, d).to(torch.bfloat16), lse


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "rope":
        return _rope(s, s["q"]), _rope(s, s["k"])
    if op == "rope_train":
        return _rope(s, s["q"]), _rope(s, s["k"]), _rope(s, s["gq"], -1.0), _rope(s, s["gk"], -1.0)
    if op == "append":
        _append(s)
        return s["kc"], s["vc"]
    if op == "decode":
        return _decode(s, s["q"])
    _append(s)
    q = _turn(s, s["q"]).to(torch.bfloat16)
    return (*_decode(s, q), s["kc"], s["vc"])


# ---- the framework's calls -------------------------------------------------------------------------------------------

def _own(s):
    eba, op = s["eba"], s["case"]["op"]
    if op == "rope":
        return eba.rope_fwd(s["q"], s["k"], s["pos"], s["plan"])
    if op == "rope_train":
        q, k = eba.rope(s["q"], s["k"], s["pos"], s["plan"])
        gq, gk = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["gq"], s["gk"]))
        return q, k, gq, gk
    if op == "append":
        eba.cache_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["cu"], rope=s["plan"], positions=s["pos"])
        return s["kc"], s["vc"]
    if op == "decode":
        return eba.decode(s["cache"], s["q"], s["table"], s["lens"])
    eba.cache_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], rope=s["plan"], positions=s["pos"])
    o, lse = eba.decode(s["cache"], s["q"], s["table"], s["lens"], rope=s["plan"], positions=s["pos"])
    return o, lse, s["kc"], s["vc"]


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    op, d, hkv = case["op"], case["d"], case["Hkv"]
    size = 1 if case.get("cache") == "e4m3" else 2
    nbytes = flops = 0
    if op in ("rope", "rope_train"):
        heads = case["B"] * case["L"] * (case["H"] + hkv)
        passes = 2 if op == "rope_train" else 1
        nbytes = passes * heads * d * 4 + 4 * case["L"] * len(_axes(case))
        flops = passes * heads * sum(_axes(case)) * 6
    if op in ("append", "step"):
        t = case["B"] * case.get("new", 1)
        nbytes += t * hkv * d * 2 * (2 + size) + 4 * t * (len(_axes(case)) + 1)
        flops += t * hkv * sum(_axes(case)) * 6
    if op in ("decode", "step"):
        n = sum(_lens(case))
        nbytes += n * hkv * d * 2 * size + case["B"] * case["H"] * (d * 4 + 4) + 4 * sum(-(-x // case["page"]) for x in _lens(case))
        flops += 4 * n * case["H"] * d
    return {"bytes": nbytes, "flops": flops}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def _exact_turn(case, pos, x, sign=1.0):
    """Pair by pair as complex numbers: (a + ib) e^(i sign angle); x [tokens, heads, d], pos [axes, tokens]."""
    f, a = _frequencies(case)
    r = len(f)
    first = list(range(r)) if case["pairing"] == "half" else list(range(0, 2 * r, 2))
    second = [i + r for i in first] if case["pairing"] == "half" else [i + 1 for i in first]
    y = x.detach().double().clone()
    angle = sign * torch.stack([pos[i].double() * w for w, i in zip(f, a)], -1)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "rope_train"):
        def whole(x, sign):
            if case["layout"] == "thd":
                return _exact_turn(case, s["pos"], x, sign)
            return torch.stack([_exact_turn(case, s["pos"], y.transpose(0, 1), sign).transpose(0, 1) for y in x])

        out = [whole(s["q"], 1.0), whole(s["k"], 1.0)]
        return out + [whole(s["gq"], -1.0), whole(s["gk"], -1.0)] if op == "rope_train" else out
    ks, vs = _scales(case)
    lens, page = _lens(case), case["page"]
    kc, vc = s["kc"].double(), s["vc"].double()
    table = s["table"].tolist()
    if op in ("append", "step"):
        new = case.get("new", 1)
        k, v = _exact_turn(case, s["pos"], s["k"]) / ks, s["v"].double() / vs
        if case["cache"] == "e4m3":
            k, v = k.clamp(-448, 448), v.clamp(-448, 448)
        if op == "step":  # the attention reads what the cache holds, and the rotated query in its own type
            k, v = k.to(s["kc"].dtype).double(), v.to(s["vc"].dtype).double()
        for b, n in enumerate(lens):
            at = list(range(n - new, n))
            pages, slots = [table[b][p // page] for p in at], [p % page for p in at]
            kc[pages, slots], vc[pages, slots] = k[b * new:(b + 1) * new], v[b * new:(b + 1) * new]
    if op == "append":
        return kc, vc
    group = case["H"] // case["Hkv"]
    q = s["q"].double() if op == "decode" else _exact_turn(case, s["pos"], s["q"]).to(torch.bfloat16).double()
    o = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n:
            pages = table[b][: -(-n // page)]
            k, v = (ks * kc[pages].flatten(0, 1)[:n], vs * vc[pages].flatten(0, 1)[:n])
            for h in range(case["Hkv"]):
                mine = slice(h * group, (h + 1) * group)
                x = q[b, mine] @ k[:, h].t() / math.sqrt(case["d"])
                lse[b, mine] = torch.logsumexp(x, -1)
                o[b, mine] = torch.softmax(x, -1) @ v[:, h]
    return (o, lse) if op == "decode" else (o, lse, kc, vc)
