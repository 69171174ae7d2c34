"""Work for the paged K/V cache held in 4 bits: the plan of a step (block table, slot map and
positions from the requests' lengths), the append of a step's keys and values, reading them back, and
the gated attention of the step's tokens through the block table.

``listed()`` gives the cases, ``draw()`` more of the same ranges, ``prepare()`` what a program holds
before the call, ``run()`` one call (the plain torch form, or with ``own`` the library's), ``exact()``
the definition in 64 bits and ``work()`` the bytes and operations a call cannot do without.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64           # tokens of a page
GROUP = 16          # columns of a token that share a scale
E4M3_MAX = 448.0
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------------------------------- cases
def _pages(name, **kw):
    c = dict(name=name, op="pages", B=1, new=1, every=1, tokens=64)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", B=1, new=1, Hkv=8, d=128, kind="e2m1", tokens=64, exp=-4)
    c.update(kw)
    return c


def _read(name, **kw):
    c = dict(name=name, op="read", B=1, Hkv=8, d=128, kind="e2m1", tokens=64, exp=-4)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(name=name, op="attend", B=1, new=1, vary=False, Hq=32, Hkv=8, d=128, kind="e2m1", gate="none", d_model=0,
             tokens=64, ragged=False, exp=-4)
    c.update(kw)
    return c


def listed():
    return [
        # the plan of a decoding step: 64 sequences, a token each, now and then one that needs a page
        _pages("pages_step_B64", B=64, tokens=8192),
        # a step that mixes 248 decoding sequences with eight pieces of prompt
        _pages("pages_mixed_B256", B=256, new=1023, every=32, tokens=4096),
        # one decoding step of 64 sequences, 8 K/V heads: latency
        _append("append4_step_B64", B=64, tokens=2048),
        # prompts of four sequences, integers
        _append("append4_prompt_L8190", B=4, new=8190, kind="int4"),
        # pieces of a few dozen tokens that start anywhere, 64-wide heads
        _append("append4_pieces_L77", B=37, new=77, Hkv=5, d=64, tokens=1000),
        # a conversation's context read back for the next piece of its prompt
        _read("read4_T1000", tokens=1000, kind="int4"),
        # three long contexts, two K/V heads
        _read("read4_T32767", B=3, Hkv=2, tokens=32767),
        # one short sequence without a gate: the latency of a single user's step
        _attend("attend4_B1_T1000", tokens=1000, kind="int4"),
        # the decode workload of 64 sequences of 8192 tokens with the elementwise gate, now against 4 bits
        _attend("attend4_B64_T8192", B=64, gate="elementwise", d_model=4096, tokens=8192),
        # 24 sequences of unequal lengths up to 32k, two K/V heads, integers, headwise gate
        _attend("attend4_ragged_T32767", B=24, Hq=16, Hkv=2, kind="int4", gate="headwise", d_model=2048, tokens=32767,
                ragged=True),
        # up to five drafted tokens of seven sequences checked at once, 64-wide heads without sharing
        _attend("attend4_draft_L5", B=7, new=5, vary=True, Hq=16, Hkv=16, d=64, tokens=4099, ragged=True),
        # a single very long sequence: few rows, the long axis split
        _attend("attend4_B1_T131072", Hq=16, Hkv=2, tokens=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["pages", "append", "append", "read", "attend", "attend", "attend"])
    d, kind, exp = rng.choice([64, 128, 128]), rng.choice(["int4", "e2m1"]), rng.randint(-6, 0)
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "pages":
        B = _log(rng, 1, 1024)
        return _pages("", B=B, new=_log(rng, 1, max(1, 65536 // B)), every=rng.choice([1, 1, 7, 32]),
                      tokens=_log(rng, 1, 16384))
    if op == "append":
        B = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, min(32768, 33_000_000 // (B * Hkv * d))))
        return _append("", B=B, new=new, Hkv=Hkv, d=d, kind=kind, exp=exp, tokens=_log(rng, 1, 4096))
    if op == "read":
        B = _log(rng, 1, 16)
        return _read("", B=B, Hkv=Hkv, d=d, kind=kind, exp=exp,
                     tokens=_log(rng, 1, max(1, min(32768, 33_000_000 // (B * Hkv * d)))))
    G = rng.choice([1, 2, 4, 7, 8])
    B, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
    gate = rng.choice(["none", "headwise", "elementwise"])
    if gate == "headwise" and Hkv * G % 8 != 0:
        gate = "elementwise"
    tokens = _log(rng, new, max(new + 1, min(131072, 536_000_000 // (B * Hkv * d))))
    return _attend("", B=B, new=new, vary=rng.random() < 0.5, Hq=Hkv * G, Hkv=Hkv, d=d, kind=kind, exp=exp, gate=gate,
                   d_model=0 if gate == "none" else rng.choice([1024, 2048, 4096]), tokens=tokens,
                   ragged=rng.random() < 0.6)


def _batch(case):
    """(tokens before the step, new tokens) of each sequence, by the case alone."""
    B, op = case["B"], case["op"]
    part = [math.modf((b + 1) * 0.6180339887)[0] for b in range(B)]
    if op == "read":
        return [0] * B, [max(1, int(case["tokens"] * (0.5 + 0.5 * p))) if b else case["tokens"]
                         for b, p in enumerate(part)]
    if op == "pages":
        # every so-many-th sequence brings that many tokens, the others one
        return ([int(case["tokens"] * p) for p in part],
                [case["new"] if b % case["every"] == 0 else 1 for b in range(B)])
    if op == "append":
        held = [int(case["tokens"] * (0.2 + 0.8 * p)) for p in part]
        return ([0] * B if case["new"] > 1000 else held), [case["new"]] * B
    new = [1 + (7 * b + case["new"] - 1) % case["new"] if case["vary"] else case["new"] for b in range(B)]
    top = max(0, case["tokens"] - case["new"])
    held = [int(top * (0.1 + 0.9 * p)) if case["ragged"] else top for p in part]
    held[0] = top
    return held, new


def _pages_of(tokens):
    return -(-tokens // PAGE)


# -------------------------------------------------------------------------------- what a call needs
def work(case):
    held, new = _batch(case)
    N, op = sum(new), case["op"]
    if op == "pages":
        fresh = sum(_pages_of(h + n) - _pages_of(h) for h, n in zip(held, new))
        # lengths and counts in, offsets and grants out, a slot and a position for each token, page numbers
        return {"bytes": 16 * case["B"] + 12 * N + 8 * fresh, "flops": 4 * N + 16 * case["B"]}
    row = case["Hkv"] * case["d"]
    if op == "append":
        return {"bytes": N * (4 * row + row * 9 // 8 + 8), "flops": 2 * N * row * 3}
    if op == "read":
        return {"bytes": N * (4 * row + row * 9 // 8 + 8), "flops": 2 * N * row * 2}
    T = [h + n for h, n in zip(held, new)]
    cols = {"none": 0, "headwise": case["Hq"], "elementwise": case["Hq"] * case["d"]}[case["gate"]]
    b = sum(T) * row * 9 // 8 + 4 * sum(_pages_of(t) for t in T) + 2 * N * case["Hq"] * case["d"] * 2
    b += 2 * case["d_model"] * cols + (2 * N * case["d_model"] if cols else 0)
    f = sum(4 * n * case["Hq"] * case["d"] * t for n, t in zip(new, T)) + 2 * N * case["d_model"] * cols
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------------------- the pool's own bytes
# A page of one head is 72 d bytes: 64 d / 2 of key codes, 64 d / 16 of key scales, the same of the
# values. Keys lie token by token, values in tiles of 16 tokens x 16 columns, one 32-bit word to a lane
# of the tensor core's operand; in both a byte holds two codes of one token.
def _pack(k, ks, v, vs, kind):
    """Codes (uint8 below 16) k, v [..., 64, d] and scales (e4m3 bytes) [..., 64, d / 16] -> [..., 72 d]."""
    d, lead = k.shape[-1], k.shape[:-2]
    n = len(lead)

    def turn(x, *order):
        return x.permute(*range(n), *(n + i for i in order))

    if kind == "int4":      # [token, j / 2, j % 2, t, pair, side] -> [token, t, j / 2, side, j % 2, pair]
        k = turn(k.reshape(*lead, PAGE, d // 32, 2, 4, 2, 2), 0, 3, 1, 5, 2, 4)
    else:                   # [token, j, t, pair, side] -> [token, t, j, pair, side]
        k = turn(k.reshape(*lead, PAGE, d // 16, 4, 2, 2), 0, 2, 1, 3, 4)
    # [tile, y, t, z, quad, i, x, g] -> [tile, quad, g, t, i, (z, y) or (y, z), x]
    v = v.reshape(*lead, 4, 2, 4, 2, d // 64, 4, 2, 8)
    v = turn(v, 0, 4, 7, 2, 5, 3, 1, 6) if kind == "int4" else turn(v, 0, 4, 7, 2, 5, 1, 3, 6)
    # [tile, y, t, z, i] -> [tile, t, i, y, z]
    vs = turn(vs.reshape(*lead, 4, 2, 4, 2, d // 16), 0, 2, 4, 1, 3)

    def pairs(x):
        return (x[..., 0] | x[..., 1] << 4).reshape(*lead, -1)

    return torch.cat((pairs(k), ks.reshape(*lead, -1), pairs(v), vs.reshape(*lead, -1)), -1)


def _unpack(page, kind):
    """[..., 72 d] -> codes k, v [..., 64, d] and scales (bytes) ks, vs [..., 64, d / 16]."""
    d, lead = page.shape[-1] // 72, page.shape[:-1]
    n = len(lead)

    def turn(x, *order):
        return x.permute(*range(n), *(n + i for i in order))

    def nibbles(x):
        return torch.stack((x & 15, x >> 4), -1)

    k, ks, v, vs = page.split((32 * d, 4 * d, 32 * d, 4 * d), -1)
    if kind == "int4":
        k = turn(nibbles(k).reshape(*lead, PAGE, 4, d // 32, 2, 2, 2), 0, 2, 4, 1, 5, 3)
    else:
        k = turn(nibbles(k).reshape(*lead, PAGE, 4, d // 16, 2, 2), 0, 2, 1, 3, 4)
    v = nibbles(v).reshape(*lead, 4, d // 64, 8, 4, 4, 2, 2, 2)      # [tile, quad, g, t, i, a, b, x]
    v = turn(v, 0, 6, 3, 5, 1, 4, 7, 2) if kind == "int4" else turn(v, 0, 5, 3, 6, 1, 4, 7, 2)
    vs = turn(vs.reshape(*lead, 4, 4, d // 16, 2, 2), 0, 3, 1, 4, 2)
    return (k.reshape(*lead, PAGE, d), ks.reshape(*lead, PAGE, d // 16), v.reshape(*lead, PAGE, d),
            vs.reshape(*lead, PAGE, d // 16))


def _code_values(codes, kind):
    if kind == "int4":
        return codes.float() - 8
    lut = torch.tensor(E2M1 + [-x for x in E2M1], device=codes.device)
    return lut.index_select(0, codes.reshape(-1).int()).reshape(codes.shape)


def _values(codes, scales, kind, exp):
    """What codes [..., d] and scale bytes [..., d / 16] stand for, in float32."""
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * 2.0 ** exp
    return (_code_values(codes, kind).unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _quantise(x, kind, exp):
    """x [..., d] -> codes (uint8 below 16) and scale bytes, in float32 (its quotients decide as exact ones)."""
    x = x.float().unflatten(-1, (-1, GROUP))
    top = 6.0 if kind == "e2m1" else 7.0
    scale = (x.abs().amax(-1) * 2.0 ** -exp / top).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    y = x / (scale.float() * 2.0 ** exp)[..., None]
    if kind == "int4":
        codes = torch.where(y.isnan(), 0.0, y.round().clamp(-7, 7)).to(torch.int8) + 8
    else:
        a = y.abs()
        codes = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
        codes = torch.where(y.isnan(), 0, codes | (y.signbit().to(torch.uint8) << 3))
        codes = torch.where(scale.float()[..., None] == 0, 0, codes)
    if kind == "int4":
        codes = torch.where(scale.float()[..., None] == 0, 8, codes)
    return codes.to(torch.uint8).flatten(-2), scale.view(torch.uint8)


# ------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(g, n_pages, Hkv, d, kind, exp):
    """Pages of normal keys and values, held as the append would."""
    pool = torch.empty((n_pages, Hkv, 72 * d), dtype=torch.uint8, device="cuda")
    step = max(1, 2 ** 26 // (Hkv * PAGE * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        kv = [_quantise(torch.randn((n, Hkv, PAGE, d), generator=g, device="cuda", dtype=torch.bfloat16), kind, exp)
              for _ in range(2)]
        pool[i:i + n] = _pack(*kv[0], *kv[1], kind)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    held, new = _batch(case)
    B, N, op = case["B"], sum(new), case["op"]
    ends = [h + n for h, n in zip(held, new)]
    most = max(_pages_of(e) for e in ends)
    in_use = sum(_pages_of(h if op == "pages" else e) for h, e in zip(held, ends))
    n_pages = sum(_pages_of(e) for e in ends) + 8
    order = torch.randperm(n_pages, generator=g, device="cuda").int()        # a pool in use: pages lie anywhere
    table = torch.full((B, most), -1, dtype=torch.int32)
    at, host = 0, order.cpu()
    for b in range(B):
        n = _pages_of(held[b] if op == "pages" else ends[b])
        table[b, :n] = host[at:at + n]
        at += n
    s["table"], s["lens"], s["new"] = table.cuda(), _ints(held), _ints(new)
    if op == "pages":
        s["free"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        s["free"][:n_pages - in_use] = order[in_use:]
        s["n_free"] = _ints([n_pages - in_use])
        s["N"] = N
        return s
    d, Hkv = case["d"], case["Hkv"]
    s["pool"] = _pool(g, n_pages, Hkv, d, case["kind"], case["exp"])
    if op in ("append", "read"):
        pos = np.concatenate([np.arange(h, e) for h, e in zip(held, ends)])
        row = np.repeat(np.arange(B), new)
        s["slots"] = torch.from_numpy(table.numpy()[row, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE).cuda()
    if op == "append":
        # keys come from the rotary positions' kernel, values lie in the packed projection's output; a
        # few columns of the keys are several times larger than the others, as trained keys' are
        loud = torch.where(torch.rand((Hkv, d), generator=g, device="cuda") < 0.03, 6.0, 1.0)
        s["K"] = (_randn(g, N, Hkv, d) * loud).bfloat16()
        s["V"] = _randn(g, N, 2 * Hkv * d).bfloat16()[:, Hkv * d:].unflatten(-1, (Hkv, d))
    if op == "attend":
        Hq, dm = case["Hq"], case["d_model"]
        s["cu"] = _ints(np.concatenate(([0], np.cumsum(new))).tolist())
        s["Q"] = (1.5 * _randn(g, N, Hq, d)).bfloat16()
        s["X"] = s["W_g"] = None
        if case["gate"] != "none":
            cols = Hq if case["gate"] == "headwise" else Hq * d
            s["X"] = _randn(g, N, dm).bfloat16()
            s["W_g"] = (0.02 * _randn(g, dm, cols)).bfloat16()
    return s


# -------------------------------------------------------------------------- the library's own calls
def _own(s):
    from gated_softmax_attention_gb300 import binding as gb
    c = s["case"]
    if c["op"] == "pages":
        step = gb.pages_step(s["lens"], s["new"], s["table"], s["free"], s["n_free"], s["N"])
        return {"cu": step.cu, "granted": step.granted, "slots": step.slots, "positions": step.positions,
                "n_free": step.n_free, "table": s["table"]}
    cache = s.get("handle")
    if cache is None:           # the handle that a program keeps beside its pool
        cache = s["handle"] = gb.Cache4(s["pool"], c["kind"], k_exp=c["exp"], v_exp=c["exp"])
    if c["op"] == "append":
        # (the pool's bytes: the definition says what each one is, so they are compared as whole numbers)
        gb.cache4_append(cache, s["K"], s["V"], s["slots"])
        return s["pool"]
    if c["op"] == "read":
        return gb.cache4_read(cache, s["slots"])
    return gb.gated_sdpa_cache4(s["X"], s["Q"], cache, s["table"], s["lens"], s["cu"], s["W_g"], gate=c["gate"],
                                max_new=c["new"])


# ----------------------------------------------------------------------------------- the plain form
def _plain_pages(s):
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"]
    B, width = table.shape
    end = lens + new
    have = (lens + PAGE - 1) // PAGE
    need = (end + PAGE - 1) // PAGE - have
    run_up = need.cumsum(0)
    count = s["n_free"].long()
    granted = (need == 0) | (run_up <= count)
    before = run_up - need
    j = torch.arange(width, device="cuda")
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None]) & granted[:, None]
    index = (count - 1 - before[:, None] - (j - have[:, None])).clamp(0, len(s["free"]) - 1)
    table.copy_(torch.where(fresh, s["free"][index], table))
    cu = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    i = torch.arange(s["N"], device="cuda")
    b = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=B - 1)
    pos = lens[b] + i - cu[b]
    slots = table[b, (pos // PAGE).clamp(max=width - 1)].long() * PAGE + pos % PAGE
    slots = torch.where(granted[b] & (i < cu[-1]), slots, -1)
    return {"cu": cu.int(), "granted": torch.where(granted, new, 0).int(), "slots": slots, "positions": pos.int(),
            "n_free": (count - torch.where(granted, need, 0).sum()).int(), "table": table}


def _plain_append(s):
    c, pool, slots = s["case"], s["pool"], s["slots"]
    d, kind = c["d"], c["kind"]
    # the bytes of the new tokens alone, each at its place in a page of its own kind
    (kc, ks), (vc, vs) = _quantise(s["K"], kind, c["exp"]), _quantise(s["V"], kind, c["exp"])
    where = _places(d, kind)
    page, at = slots // PAGE, slots % PAGE
    head = torch.arange(c["Hkv"], device="cuda")[:, None]
    flat = (page[:, None, None] * c["Hkv"] + head) * (72 * d) + where[at][:, None]      # [N, Hkv, bytes]
    pool.view(-1)[flat] = torch.cat((_bytes(kc, "k", kind), ks, _bytes(vc, "v", kind), vs), -1)
    return pool


def _places(d, kind):
    """[64, 9 d / 8]: which bytes of a page are token i's, in the order of _bytes and the scales."""
    mark = torch.arange(PAGE, device="cuda")[:, None]
    zero = torch.zeros((PAGE, d // 16), dtype=torch.int64, device="cuda")
    half = d // 2
    out = torch.empty((PAGE, d + d // 8), dtype=torch.int64, device="cuda")
    at = torch.arange(72 * d, device="cuda")
    out[:, :half] = (mark * half + torch.arange(half, device="cuda"))
    out[:, half:half + d // 16] = 32 * d + mark * (d // 16) + torch.arange(d // 16, device="cuda")
    # values: the tile's words in order, the token's byte in each
    tile, y, t, z = mark // 16, mark // 8 % 2, mark // 2 % 4, mark % 2
    byte = 2 * z + y if kind == "int4" else 2 * y + z
    w = torch.arange(half, device="cuda")                                     # [quad, g, i]
    quad, g, i = w // 32, w // 4 % 8, w % 4
    out[:, half + d // 16:d + d // 16] = 36 * d + (((tile * (d // 64) + quad) * 32 + g * 4 + t) * 4 + i) * 4 + byte
    j = torch.arange(d // 16, device="cuda")
    out[:, d + d // 16:] = 68 * d + ((tile * 4 + t) * (d // 16) + j) * 4 + 2 * y + z
    return out


def _bytes(codes, which, kind):
    """A token's codes [..., d] as the bytes it has in a page, [..., d / 2]."""
    d, lead = codes.shape[-1], codes.shape[:-1]
    if which == "v":        # [quad, i, x, g] -> [quad, g, i, x]
        x = codes.reshape(*lead, d // 64, 4, 2, 8).permute(*range(len(lead)), -4, -1, -3, -2)
    elif kind == "int4":    # [j / 2, j % 2, t, pair, side] -> [t, j / 2, side, j % 2, pair]
        x = codes.reshape(*lead, d // 32, 2, 4, 2, 2).permute(*range(len(lead)), -3, -5, -1, -4, -2)
    else:                   # [j, t, pair, side] -> [t, j, pair, side]
        x = codes.reshape(*lead, d // 16, 4, 2, 2).permute(*range(len(lead)), -3, -4, -2, -1)
    return (x[..., 0] | x[..., 1] << 4).reshape(*lead, d // 2)


def _plain_read(s):
    c, slots = s["case"], s["slots"]
    where = _places(c["d"], c["kind"])
    d, half = c["d"], c["d"] // 2
    head = torch.arange(c["Hkv"], device="cuda")[:, None]
    flat = ((slots // PAGE)[:, None, None] * c["Hkv"] + head) * (72 * d) + where[slots % PAGE][:, None]
    x = s["pool"].view(-1)[flat]
    kb, ks, vb, vs = x.split((half, d // 16, half, d // 16), -1)
    lead = kb.shape[:-1]
    n = range(len(lead))
    kb, vb = (torch.stack((b & 15, b >> 4), -1) for b in (kb, vb))
    if c["kind"] == "int4":
        k = kb.reshape(*lead, 4, d // 32, 2, 2, 2).permute(*n, -4, -2, -5, -1, -3)
    else:
        k = kb.reshape(*lead, 4, d // 16, 2, 2).permute(*n, -3, -4, -2, -1)
    v = vb.reshape(*lead, d // 64, 8, 4, 2).permute(*n, -4, -2, -1, -3)
    return tuple(_values(y.reshape(*lead, d), sc, c["kind"], c["exp"]).bfloat16() for y, sc in ((k, ks), (v, vs)))


def _plain_attend(s):
    c, lens, cu = s["case"], s["lens"].long(), s["cu"].long()
    Hq, Hkv, d, Lq = c["Hq"], c["Hkv"], c["d"], c["new"]
    G = Hq // Hkv
    k, ks, v, vs = _unpack(s["pool"][s["table"].long().clamp(min=0)].transpose(1, 2), c["kind"])   # [B, Hkv, pages, ..]
    k = _values(k, ks, c["kind"], c["exp"]).flatten(2, 3)                    # [B, Hkv, S, d]
    v = _values(v, vs, c["kind"], c["exp"]).flatten(2, 3)
    i = torch.arange(Lq, device="cuda")
    rows = cu[:-1, None] + i                                                 # [B, Lq], some past the sequence's
    real = rows < cu[1:, None]
    rows = torch.where(real, rows, cu[:-1, None])
    q = s["Q"].float()[rows].unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, Hkv, Lq * G, d]
    score = q @ k.transpose(-1, -2) / math.sqrt(d)
    at = torch.arange(k.shape[2], device="cuda")
    unseen = at > (lens[:, None] + i).repeat_interleave(G, 1)[..., None]     # [B, Lq * G, S]
    past = (at >= (lens + cu[1:] - cu[:-1])[:, None])[:, None, :, None]      # what lies behind a sequence is not looked at
    v = torch.where(past, 0.0, v)
    score = score.masked_fill(unseen[:, None] | past.transpose(-1, -2), -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    o = o.unflatten(2, (Lq, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)         # [B, Lq, Hq, d]
    out = torch.empty((len(s["Q"]), Hq, d), device="cuda")
    flat = torch.where(real, rows, len(out))                                 # (a row behind the last takes the others')
    out = torch.cat((out, out[:1]))
    out[flat.flatten()] = o.flatten(0, 1)
    out = out[:-1]
    if c["gate"] != "none":
        sig = 1 / (1 + torch.exp(-(s["X"].float() @ s["W_g"].float())))
        out = out * (sig[..., None] if c["gate"] == "headwise" else sig.unflatten(-1, (Hq, d)))
    return out.to(s["Q"].dtype)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"pages": _plain_pages, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[op](state)


# --------------------------------------------------------------------------- the definition, 64 bits
def _where_exact(d, kind):
    """Of every code of a page, (token, column) -> byte and shift, and of every scale -> byte; written
    out place by place."""
    k, v = np.zeros((PAGE, d, 2), dtype=np.int64), np.zeros((PAGE, d, 2), dtype=np.int64)
    ks, vs = np.zeros((PAGE, d // 16), dtype=np.int64), np.zeros((PAGE, d // 16), dtype=np.int64)
    for n in range(PAGE):
        for col in range(d):
            j, r = col // 16, col % 16
            lane, pair, side = r // 4, r // 2 % 2, r % 2
            base = n * d // 2 + lane * d // 8
            if kind == "e2m1":
                k[n, col] = base + 2 * j + pair, 4 * side
            else:
                bit = 16 * side + 4 * (2 * (j % 2) + pair)
                k[n, col] = base + 4 * (j // 2) + bit // 8, bit % 8
            g, x = r % 8, r // 8
            t, z, y = n % 8 // 2, n % 2, n % 16 // 8
            word = ((n // 16 * (d // 64) + j // 4) * 32 + 4 * g + t) * 4 + j % 4
            if kind == "e2m1":
                v[n, col] = 36 * d + 4 * word + 2 * y + z, 4 * x
            else:
                bit = 16 * z + 4 * (x + 2 * y)
                v[n, col] = 36 * d + 4 * word + bit // 8, bit % 8
        for j in range(d // 16):
            ks[n, j] = 32 * d + n * d // 16 + j
            vs[n, j] = 68 * d + ((n // 16 * 4 + n % 8 // 2) * (d // 16) + j) * 4 + 2 * (n % 16 // 8) + n % 2
    return [torch.from_numpy(x).cuda() for x in (k, ks, v, vs)]


def _held_exact(page, d, kind, exp, places):
    """Keys and values of whole pages [n, 72 d] as float64 [n, 64, d]."""
    k, ks, v, vs = places
    table = torch.tensor([float(x - 8) for x in range(16)] if kind == "int4" else E2M1 + [-x for x in E2M1],
                         dtype=torch.float64, device="cuda")
    byte = torch.arange(256, device="cuda")
    e, m = byte % 128 // 8, (byte % 8).double()
    sc = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    sc = torch.where(byte % 128 == 127, math.nan, sc * torch.where(byte > 127, -1.0, 1.0)) * 2.0 ** exp
    out = []
    for c, s in ((k, ks), (v, vs)):
        codes = page[:, c[..., 0]].long() >> c[..., 1] & 15
        out.append(table[codes] * sc[page[:, s].long()].repeat_interleave(16, -1))
    return out


def _codes_exact(x, kind, exp):
    """A row's 16 float64 numbers [..., 16] -> codes and the scale's byte [...]."""
    top = 6.0 if kind == "e2m1" else 7.0
    want = x.abs().amax(-1) / top / 2.0 ** exp
    grid = torch.tensor([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)
                         ][:127], dtype=torch.float64, device="cuda")
    up = torch.searchsorted(grid, want.contiguous()).clamp(max=126)          # the least not below
    down = (up - 1).clamp(min=0)
    to_up, to_down = (grid[up] - want).abs(), (want - grid[down]).abs()
    byte = torch.where((to_up < to_down) | ((to_up == to_down) & (up % 2 == 0)), up, down)
    step = grid[byte] * 2.0 ** exp
    y = torch.where(step[..., None] > 0, x / step[..., None], torch.zeros_like(x))
    if kind == "int4":
        return (torch.round(y).clamp(-7, 7) + 8).long(), byte
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    off = (y.abs().clamp(max=6.0)[..., None] - mag).abs()
    best = off.amin(-1, keepdim=True)
    near = off == best
    even = near & (torch.arange(8, device="cuda") % 2 == 0)
    code = torch.where(even.any(-1), even.long().argmax(-1), near.long().argmax(-1))
    negative = torch.signbit(x) & (step[..., None] > 0)
    return code + 8 * negative.long(), byte


def exact(case, seed):
    c = case
    held, new = _batch(c)
    if c["op"] == "pages":
        s = prepare(c, seed)
        table, free, left = s["table"].tolist(), s["free"].tolist(), int(s["n_free"])
        cu, granted, slots, positions, asked, taken = [0], [], [], [], 0, 0
        for b, (h, n) in enumerate(zip(held, new)):
            need = _pages_of(h + n) - _pages_of(h)
            asked += need
            ok = need == 0 or asked <= left
            for k in range(need if ok else 0):
                table[b][_pages_of(h) + k] = free[left - 1 - (asked - need) - k]
            taken += need if ok else 0
            granted.append(n if ok else 0)
            cu.append(cu[-1] + n)
            positions += range(h, h + n)
            slots += [table[b][p // PAGE] * PAGE + p % PAGE if ok else -1 for p in range(h, h + n)]
        return {"cu": _ints(cu), "granted": _ints(granted), "slots": torch.tensor(slots, device="cuda"),
                "positions": _ints(positions), "n_free": _ints([left - taken]), "table": _ints(table)}
    d, kind, Hkv = c["d"], c["kind"], c["Hkv"]
    s = prepare(c, seed)
    places = _where_exact(d, kind)
    if c["op"] == "append":
        pool = s["pool"].clone()
        where, slots = places, s["slots"]
        page, at = slots // PAGE, slots % PAGE
        base = (page[:, None] * Hkv + torch.arange(Hkv, device="cuda")) * (72 * d)           # [N, Hkv]
        flat = pool.view(-1)
        for x, (code_at, scale_at) in ((s["K"], where[:2]), (s["V"], where[2:])):
            for j in range(d // 16):                                          # (column by column: two share a byte)
                codes, byte = _codes_exact(x[..., 16 * j:16 * j + 16].double(), kind, c["exp"])
                flat[base + scale_at[at, j][:, None]] = byte.to(torch.uint8)
                for r in range(16):
                    w, sh = code_at[at, 16 * j + r].unbind(-1)
                    to, sh = base + w[:, None], sh[:, None]
                    flat[to] = ((flat[to].long() & ~(15 << sh)) | codes[..., r] << sh).to(torch.uint8)
        return pool
    if c["op"] == "read":
        page, at = s["slots"] // PAGE, s["slots"] % PAGE
        rows = [[], []]
        for h in range(Hkv):
            for i in range(0, len(page), 4096):
                part = page[i:i + 4096]
                each, index = part.unique(return_inverse=True)
                for out, x in zip(rows, _held_exact(s["pool"][each, h], d, kind, c["exp"], places)):
                    out.append(x[index, at[i:i + 4096]])
        n = len(range(0, len(page), 4096))
        return tuple(torch.stack([torch.cat(r[h * n:(h + 1) * n]) for h in range(Hkv)], 1) for r in rows)
    o = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    G, at = c["Hq"] // Hkv, 0
    for b, (start, n) in enumerate(zip(held, new)):
        T = start + n
        pages = s["table"][b, :_pages_of(T)].long()
        for h in range(Hkv):
            k, v = (x.flatten(0, 1)[:T] for x in _held_exact(s["pool"][pages, h], d, kind, c["exp"], places))
            for i in range(n):
                q = s["Q"][at + i, h * G:(h + 1) * G].double()
                w = torch.softmax(q @ k[:start + i + 1].T / math.sqrt(d), -1)
                o[at + i, h * G:(h + 1) * G] = w @ v[:start + i + 1]
        at += n
    if c["gate"] != "none":
        sig = torch.sigmoid(s["X"].double() @ s["W_g"].double())
        o = o * (sig[..., None] if c["gate"] == "headwise" else sig.reshape(o.shape))
    return o
