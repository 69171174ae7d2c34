"""Work for the operators around the gated attention: queries and keys normalised per head and
rotated by position (forward and backward), keys and values appended to a cache held in 8 bits, and
the gated attention of new tokens against that cache.

``listed()`` gives the cases, ``draw()`` more of the same ranges, ``prepare()`` what a program holds
before the call, ``run()`` one call (the plain torch form, or with ``own`` the library's), ``exact()``
the definition in 64 bits and ``work()`` the bytes and operations a call cannot do without.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64          # tokens that share one scale of the 8-bit cache
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------- cases
def _rope(name, **kw):
    c = dict(name=name, op="rope", B=1, L=1, Hq=16, Hkv=16, d=128, dtype="bf16", norm=True, layout="half",
             rotary=128, scaling="none", factor=1.0, orig_len=4096, far=0)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", B=1, L=1, Hkv=8, d=128, kind="int8", start=0)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(name=name, op="attend", B=1, Lq=1, Hq=32, Hkv=8, d=128, kind="int8", gate="none", d_model=0, tokens=64,
             ragged=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of 64 sequences, 32/8 heads, each at its own position: latency
        _rope("rope_step_B64", B=64, L=1, Hq=32, Hkv=8, far=8192),
        # the prompt of a GQA 32/4 layer at its training context
        _rope("rope_gqa_L4096", B=1, L=4096, Hq=32, Hkv=4),
        # float32, odd lengths, a quarter of a 64-wide head rotated in adjacent pairs, positions compressed linearly
        _rope("rope_f32_part_L509", B=3, L=509, Hq=16, Hkv=16, d=64, dtype="f32", layout="interleaved", rotary=16,
              scaling="linear", factor=4.0),
        # the backward of a training step of the headline layer
        _rope("rope_bwd_mha_L2048", op="rope_bwd", B=2, L=2048, Hq=16, Hkv=16),
        # the backward of the long-context stage, frequencies scaled by parts from 4096 to 32k
        _rope("rope_bwd_gqa_L32768", op="rope_bwd", B=1, L=32768, Hq=16, Hkv=2, layout="interleaved", scaling="parts",
              factor=8.0, orig_len=4096),
        # one decoding step of 64 sequences: a token each, now and then one that fills its block
        _append("append_step_B64", B=64, L=1, Hkv=8, kind="int8", start=2048),
        # prompts of four sequences into an empty e4m3 cache
        _append("append_prompt_L8190", B=4, L=8190, Hkv=8, kind="e4m3", start=0),
        # one short sequence without a gate: the latency of a single user's step
        _attend("attend_B1_T1000", B=1, Hq=32, Hkv=8, tokens=1000),
        # the decode workload of 64 sequences of 8192 tokens with the elementwise gate, now against int8
        _attend("attend_B64_T8192", B=64, Hq=32, Hkv=8, gate="elementwise", d_model=4096, tokens=8192),
        # 24 sequences of unequal lengths up to 32k, two K/V heads, e4m3, headwise gate
        _attend("attend_ragged_T32767", B=24, Hq=16, Hkv=2, kind="e4m3", gate="headwise", d_model=2048, tokens=32767,
                ragged=True),
        # five drafted tokens of seven sequences checked at once, 64-wide heads without sharing
        _attend("attend_draft_Lq5", B=7, Lq=5, Hq=16, Hkv=16, d=64, tokens=4099, ragged=True),
        # a single very long sequence: few rows, the long axis split
        _attend("attend_B1_T131072", B=1, Hq=16, Hkv=2, kind="e4m3", tokens=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    if op in ("rope", "rope_bwd"):
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 8) if Hkv * g <= 32])
        B = _log(rng, 1, 64)
        rows = 75_000_000 // (B * (Hq + Hkv) * d)
        L = _log(rng, 1, max(1, min(32768, rows)))
        scaling = rng.choice(["none", "none", "linear", "base", "parts"])
        return _rope("", op=op, B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                     norm=rng.random() < 0.8, layout=rng.choice(["half", "interleaved"]),
                     rotary=16 * rng.randint(1, d // 16), scaling=scaling,
                     factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                     far=rng.choice([0, 0, 4096, 1_000_000]))
    if op == "append":
        Hkv, B = rng.choice([1, 2, 4, 8, 16]), _log(rng, 1, 64)
        L = _log(rng, 1, max(1, min(32768, 33_000_000 // (B * Hkv * d))))
        start = _log(rng, 1, 8192) if rng.random() < 0.7 else 0
        return _append("", B=B, L=L, Hkv=Hkv, d=d, kind=rng.choice(["int8", "e4m3"]), start=start)
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 4, 7, 8])
    B, Lq = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
    gate = rng.choice(["none", "headwise", "elementwise"])
    if gate == "headwise" and Hkv * G % 8 != 0:
        gate = "elementwise"
    tokens = _log(rng, Lq, max(Lq + 1, min(131072, 536_000_000 // (B * Hkv * d))))
    return _attend("", B=B, Lq=Lq, Hq=Hkv * G, Hkv=Hkv, d=d, kind=rng.choice(["int8", "e4m3"]), gate=gate,
                   d_model=0 if gate == "none" else rng.choice([1024, 2048, 4096]), tokens=tokens,
                   ragged=rng.random() < 0.6)


def _starts(case):
    """Tokens each sequence of the batch holds before the call, by the case alone."""
    B = case["B"]
    if case["op"] == "append":
        top = case["start"]
        # (a step goes on anywhere; a long piece of prompt begins with a block)
        v = [int(top * (0.2 + 0.8 * math.modf((b + 1) * 0.6180339887)[0])) for b in range(B)]
        return v if case["L"] <= BLOCK else [x // BLOCK * BLOCK for x in v]
    top = max(0, case["tokens"] - case["Lq"])
    if not case["ragged"]:
        return [top] * B
    v = [int(top * (0.1 + 0.9 * math.modf((b + 1) * 0.6180339887)[0])) for b in range(B)]
    v[0] = top
    return v


# -------------------------------------------------------------------------------- what a call needs
def work(case):
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        es = 2 if case["dtype"] == "bf16" else 4
        n = case["B"] * case["L"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": (2 if op == "rope" else 3) * es * n, "flops": (8 if op == "rope" else 18) * n}
    row = case["Hkv"] * case["d"]
    if op == "append":
        # every new token read once as bf16, and written as 8 bits or, in the open block, as bf16
        b = f = 0
        for s in _starts(case):
            end = s + case["L"]
            closed = end // BLOCK * BLOCK
            q = max(0, closed - s // BLOCK * BLOCK)         # tokens written in 8 bits
            old = (s % BLOCK) if closed > s else 0          # ... of which these come from the open block
            b += 2 * row * (2 * case["L"] + 2 * old + q + 2 * (end - max(s, closed)))
            f += 2 * row * 4 * q
        return {"bytes": b, "flops": f}
    T = [s + case["Lq"] for s in _starts(case)]
    held = sum(T) * row
    cols = {"none": 0, "headwise": case["Hq"], "elementwise": case["Hq"] * case["d"]}[case["gate"]]
    rows = case["B"] * case["Lq"]
    b = 2 * held + 8 * sum(-(-t // BLOCK) for t in T) * case["Hkv"] + 2 * rows * case["Hq"] * case["d"] * 2
    b += 2 * case["d_model"] * cols + (2 * rows * case["d_model"] if cols else 0)
    f = 4 * case["Lq"] * (case["Hq"] // case["Hkv"]) * held + 2 * rows * case["d_model"] * cols
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------------- inputs
def _type(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _cache(g, B, Hkv, capacity, d, kind):
    """A cache of that many tokens: codes of normal keys and values and the scales that go with them."""
    n = capacity // BLOCK
    shape_k, shape_v = (B, Hkv, n, BLOCK, d), (B, Hkv, n, d, BLOCK)

    def codes(shape):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if kind == "int8":
            return (x * 31).round_().clamp_(-127, 127).to(torch.int8)
        return (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales():
        u = torch.rand((B, Hkv, n), generator=g, device="cuda")
        return (0.8 + 0.4 * u) / 31 if kind == "int8" else torch.where(u < 0.5, 2.0 ** -7, 2.0 ** -6)

    return {"k8": codes(shape_k), "v8": codes(shape_v), "k_scale": scales(), "v_scale": scales(),
            "k_tail": _randn(g, B, Hkv, 2, BLOCK, d).bfloat16(), "v_tail": _randn(g, B, Hkv, 2, d, BLOCK).bfloat16()}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    B, d, Hkv = case["B"], case["d"], case["Hkv"]
    if case["op"] in ("rope", "rope_bwd"):
        L, Hq, td = case["L"], case["Hq"], _type(case)
        # the projection's output, [Q | K | V] of each token in one row
        packed = _randn(g, B, L, (Hq + 2 * Hkv) * d).to(td)
        s["Q"] = packed[..., :Hq * d].unflatten(-1, (Hq, d))
        s["K"] = packed[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
        s["gamma_q"] = (1 + 0.1 * _randn(g, d)).to(td) if case["norm"] else None
        s["gamma_k"] = (1 + 0.1 * _randn(g, d)).to(td) if case["norm"] else None
        s["positions"] = None
        if case["far"]:
            first = torch.randint(0, case["far"], (B, 1), generator=g, device="cuda", dtype=torch.int32)
            s["positions"] = (first + torch.arange(L, device="cuda", dtype=torch.int32)).contiguous()
        if case["op"] == "rope_bwd":
            s["dQ"] = (_randn(g, B, L, Hq, d) / 8).to(td)
            s["dK"] = (_randn(g, B, L, Hkv, d) / 8).to(td)
        return s
    starts = _starts(case)
    n_new = case["L"] if case["op"] == "append" else case["Lq"]
    capacity = (max(starts) + n_new + BLOCK - 1) // BLOCK * BLOCK + BLOCK
    s["cache"] = _cache(g, B, Hkv, capacity, d, case["kind"])
    s["lens"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        s["K"] = _randn(g, B, n_new, Hkv, d).bfloat16()
        s["V"] = _randn(g, B, n_new, Hkv, d).bfloat16()
        return s
    Hq, dm = case["Hq"], case["d_model"]
    s["Q"] = (1.5 * _randn(g, B, n_new, Hq, d)).bfloat16()
    s["X"] = s["W_g"] = None
    if case["gate"] != "none":
        cols = Hq if case["gate"] == "headwise" else Hq * d
        s["X"] = _randn(g, B, n_new, dm).bfloat16()
        s["W_g"] = (0.02 * _randn(g, dm, cols)).bfloat16()
    return s


# -------------------------------------------------------------------------- the library's own calls
def _own(s):
    from gated_softmax_attention_gb300 import binding as gb
    c = s["case"]
    if c["op"] in ("rope", "rope_bwd"):
        rope = s.get("rope")
        if rope is None:        # the plan that a program makes once
            rope = s["rope"] = gb.Rope(c["rotary"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                                       orig_len=c["orig_len"])
        kw = dict(gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], norm=c["norm"], eps=EPS, rope=rope,
                  positions=s["positions"])
        if c["op"] == "rope":
            return gb.qk_norm_rope(s["Q"], s["K"], **kw)
        return gb.qk_norm_rope_bwd(s["Q"], s["K"], s["dQ"], s["dK"], **kw)
    cache = s.get("handle")
    if cache is None:           # the handle that a program keeps beside its cache
        cache = s["handle"] = gb.Cache8(**s["cache"])
    if c["op"] == "append":
        # (codes come back in the types whose values they are, int8 or float8_e4m3fn, their scales beside them)
        gb.cache8_append(cache, s["K"], s["V"], s["lens"])
        return s["cache"]
    return gb.gated_sdpa_cache8(s["X"], s["Q"], cache, s["lens"], s["W_g"], gate=c["gate"])


# ----------------------------------------------------------------------------------- the plain form
def _frequencies(c):
    """Angle per position of each pair, and the factor on cosine and sine (64 bits, on the host)."""
    rd, theta = c["rotary"], 10000.0
    i = np.arange(rd // 2, dtype=np.float64)
    w, scale = theta ** (-2.0 * i / rd), 1.0
    if c["scaling"] == "linear":
        w = w / c["factor"]
    elif c["scaling"] == "base":
        w = (theta * c["factor"] ** (rd / max(rd - 2.0, 1.0))) ** (-2.0 * i / rd)
    elif c["scaling"] == "parts":
        # pairs that turn often within the old length keep their frequency, slow ones are compressed
        at = [rd * math.log(c["orig_len"] / (turns * 2 * math.pi)) / (2 * math.log(theta)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        w = w / c["factor"] * ramp + w * (1.0 - ramp)
        scale = 0.1 * math.log(c["factor"]) + 1.0
    return w, scale


def _angles(s):
    """cos and sin [B or 1, L, 1, rotary / 2], scaled; the angles in 64 bits (far positions)."""
    c = s["case"]
    w, scale = _frequencies(c)
    p = s["positions"]
    p = torch.arange(c["L"], device="cuda")[None] if p is None else p
    a = p.double()[..., None, None] * torch.from_numpy(w).cuda()
    return (a.cos() * scale).float(), (a.sin() * scale).float()


def _pairs(x, c):
    """(first, second) members of the rotated pairs, and the columns that are not rotated."""
    h = c["rotary"] // 2
    if c["layout"] == "half":
        return x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return x[..., 0:2 * h:2], x[..., 1:2 * h:2], x[..., 2 * h:]


def _join(a, b, rest, c):
    z = torch.cat((a, b), -1) if c["layout"] == "half" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((z, rest), -1)


def _plain_rope(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, gamma):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gamma.float()
        a, b, rest = _pairs(y, c)
        return _join(a * cos - b * sin, b * cos + a * sin, rest, c).to(x.dtype)

    return one(s["Q"], s["gamma_q"]), one(s["K"], s["gamma_k"])


def _plain_rope_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, dz, gamma):
        a, b, rest = _pairs(dz.float(), c)
        dy = _join(a * cos + b * sin, b * cos - a * sin, rest, c)
        if not c["norm"]:
            return dy.to(x.dtype), None
        xf = x.float()
        r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
        xh, h = xf * r, dy * gamma.float()
        dx = r * (h - xh * (h * xh).mean(-1, keepdim=True))
        return dx.to(x.dtype), (dy * xh).sum((0, 1, 2)).to(gamma.dtype)

    dq, gq = one(s["Q"], s["dQ"], s["gamma_q"])
    dk, gk = one(s["K"], s["dK"], s["gamma_k"])
    out = {"dQ": dq, "dK": dk}
    if c["norm"]:
        out["dgamma_q"], out["dgamma_k"] = gq, gk
    return out


def _plain_quantise(x, kind):
    """x [..., 64, d] of whole blocks -> codes and scales [...]; quotients in 64 bits (values next to a border)."""
    amax = x.float().abs().amax((-1, -2))
    if kind == "int8":
        scale = amax / 127
        y = x.double() / scale.double()[..., None, None]
        return torch.where(y.isnan(), 0.0, y.round()).clamp(-127, 127).to(torch.int8), scale
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 0.0)
    y = torch.ldexp(x.float(), -e[..., None, None])
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _plain_append(s):
    c, cache, lens = s["case"], s["cache"], s["lens"].long()
    B, L = c["B"], c["L"]
    touched = (L + BLOCK - 2) // BLOCK + 1
    first = lens // BLOCK
    blk = first[:, None] + torch.arange(touched, device="cuda")              # [B, n]
    blk = torch.minimum(blk, torch.tensor(cache["k8"].shape[2] - 1, device="cuda"))
    pos = blk[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")        # [B, n, 64]
    src = (pos - lens[:, None, None]).clamp(0, L - 1)
    rows = torch.arange(B, device="cuda")[:, None]
    end = lens + L
    # the open block's buffers hold the blocks of even and odd number
    slot = torch.arange(2, device="cuda")
    last = (end - 1) // BLOCK
    ring = last[:, None] - (last[:, None] - slot) % 2                        # [B, 2]: the block each may take
    ring_pos = ring[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")  # [B, 2, 64]
    fresh = (ring_pos >= lens[:, None, None]) & (ring_pos < end[:, None, None])
    ring_src = (ring_pos - lens[:, None, None]).clamp(0, L - 1)
    closed = (blk + 1) * BLOCK <= end[:, None]                               # [B, n]
    for name, new, turn in (("k", s["K"], False), ("v", s["V"], True)):
        tail = cache[name + "_tail"]
        held = tail.transpose(-1, -2) if turn else tail                      # [B, Hkv, 2, 64, d]
        x = new[rows[..., None], src].transpose(2, 3).transpose(1, 2)        # [B, Hkv, n, 64, d]
        old = held[rows, :, blk % 2].transpose(1, 2)
        x = torch.where((pos < lens[:, None, None])[:, None, ..., None], old, x)
        codes, scale = _plain_quantise(x, c["kind"])
        codes = (codes.transpose(-1, -2) if turn else codes).transpose(1, 2).contiguous()   # [B, n, Hkv, ...]
        store, scales = cache[name + "8"], cache[name + "_scale"]
        bits = store.view(torch.int8)
        bits[rows, :, blk] = torch.where(closed[..., None, None, None], codes.view(torch.int8), bits[rows, :, blk])
        scales[rows, :, blk] = torch.where(closed[..., None], scale.transpose(1, 2), scales[rows, :, blk])
        f = new[rows[..., None], ring_src].transpose(2, 3).transpose(1, 2)   # [B, Hkv, 2, 64, d]
        held.copy_(torch.where(fresh[:, None, ..., None], f, held))
    return cache


def _plain_attend(s):
    c, cache, lens = s["case"], s["cache"], s["lens"].long()
    B, Lq, Hq, Hkv, d = c["B"], c["Lq"], c["Hq"], c["Hkv"], c["d"]
    n = cache["k8"].shape[2]
    open_blk = (lens + Lq) // BLOCK
    is_open = (torch.arange(n, device="cuda") == open_blk[:, None])[:, None, :, None, None]
    b = torch.arange(B, device="cuda")

    def values(name):
        x = cache[name + "8"].float() * cache[name + "_scale"][..., None, None]
        return torch.where(is_open, cache[name + "_tail"][b, :, open_blk % 2].float()[:, :, None], x)

    k = values("k").flatten(2, 3)                                            # [B, Hkv, S, d]
    v = values("v").transpose(-1, -2).flatten(2, 3)
    G = Hq // Hkv
    q = s["Q"].float().unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, Hkv, Lq * G, d]
    score = q @ k.transpose(-1, -2) / math.sqrt(d)
    at = torch.arange(n * BLOCK, device="cuda")
    row = torch.arange(Lq, device="cuda").repeat_interleave(G)
    unseen = at > (lens[:, None, None] + row[:, None])                       # [B, Lq * G, S]
    score = score.masked_fill(unseen[:, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    o = o.unflatten(2, (Lq, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)         # [B, Lq, Hq, d]
    if c["gate"] != "none":
        gl = s["X"].float() @ s["W_g"].float()
        sig = 1 / (1 + torch.exp(-gl))
        o = o * (sig[..., None] if c["gate"] == "headwise" else sig.unflatten(-1, (Hq, d)))
    return o.to(s["Q"].dtype)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "rope_bwd":
        return _plain_rope_bwd(state)
    return _plain_append(state) if op == "append" else _plain_attend(state)


# --------------------------------------------------------------------------- the definition, 64 bits
def _turn(c, s):
    """exp(i angle) times the scale, complex128 [B or 1, L, rotary / 2]."""
    rd, base = c["rotary"], 10000.0
    w, scale = [], 1.0
    for i in range(rd // 2):
        f = base ** (-2.0 * i / rd)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "base":
            f = (base * c["factor"] ** (rd / max(rd - 2.0, 1.0))) ** (-2.0 * i / rd)
        elif c["scaling"] == "parts":
            def where(turns):
                return rd * math.log(c["orig_len"] / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(math.floor(where(32.0)), 0), min(math.ceil(where(1.0)), rd - 1)
            u = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f * (1 - u) + f / c["factor"] * u
            scale = 0.1 * math.log(c["factor"]) + 1.0
        w.append(f)
    p = torch.arange(c["L"], device="cuda")[None] if s["positions"] is None else s["positions"]
    a = p.double()[..., None] * torch.tensor(w, dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(a, scale), a)


def _exact_forward(x, gamma, z, c):
    if c["norm"]:
        x = gamma * x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    rd = c["rotary"]
    part = x[..., :rd]
    pair = part.unflatten(-1, (2, rd // 2)).transpose(-1, -2) if c["layout"] == "half" else \
        part.unflatten(-1, (rd // 2, 2))
    t = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, :, None])
    t = t.transpose(-1, -2) if c["layout"] == "half" else t
    return torch.cat((t.flatten(-2), x[..., rd:]), -1)


def _exact_quantise(x, kind):
    """x [64, d] float64 -> codes as float64, and the scale."""
    amax = float(x.abs().max())
    if amax == 0:
        return torch.zeros_like(x), 0.0
    if kind == "int8":
        scale = float(np.float32(amax) / np.float32(127))
        return (x / scale).round().clamp(-127, 127), scale
    e = -126
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    y = x / 2.0 ** e
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)    # three bits behind the first
    return (y / step).round() * step, 2.0 ** e


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        z = _turn(c, s)
        return tuple(_exact_forward(s[n].double(), None if s[g] is None else s[g].double(), z, c)
                     for n, g in (("Q", "gamma_q"), ("K", "gamma_k")))
    if c["op"] == "rope_bwd":
        z, out = _turn(c, s), {}
        for n, g in (("Q", "gamma_q"), ("K", "gamma_k")):
            x = s[n].double().requires_grad_()
            gamma = s[g].double().requires_grad_() if c["norm"] else None
            _exact_forward(x, gamma, z, c).backward(s["d" + n].double())
            out["d" + n] = x.grad
            if c["norm"]:
                out["d" + g] = gamma.grad
        return out
    starts = _starts(c)
    cache = s["cache"]
    if c["op"] == "append":
        if c["B"] * c["Hkv"] * (c["L"] // BLOCK + 1) > 6000:
            return None         # (block by block it would take too long)
        out = {n: t.clone() for n, t in cache.items()}
        for b, start in enumerate(starts):
            end = start + c["L"]
            for h in range(c["Hkv"]):
                for n in "kv":
                    new = s[n.upper()][b, :, h]
                    tail = cache[n + "_tail"][b, h]
                    tail = tail if n == "k" else tail.transpose(-1, -2)
                    old = tail[start // BLOCK % 2][:start % BLOCK]
                    seq = torch.cat((old, new)).double()                     # from the first touched block on
                    base = start // BLOCK
                    for j in range(base, end // BLOCK):
                        q, sc = _exact_quantise(seq[(j - base) * BLOCK:(j - base + 1) * BLOCK], c["kind"])
                        q = q if n == "k" else q.T
                        out[n + "8"][b, h, j] = q.to(torch.int8) if c["kind"] == "int8" else \
                            q.float().to(torch.float8_e4m3fn)
                        out[n + "_scale"][b, h, j] = sc
                    last = (end - 1) // BLOCK
                    for j in range(max(base, last - 1), last + 1):
                        lo, hi = max(start, j * BLOCK), min(end, (j + 1) * BLOCK)
                        to = out[n + "_tail"][b, h, j % 2]
                        to = to if n == "k" else to.T
                        to[lo - j * BLOCK:hi - j * BLOCK] = new[lo - start:hi - start]
        return out
    o = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    G = c["Hq"] // c["Hkv"]
    for b, start in enumerate(starts):
        T = start + c["Lq"]
        full, rest = T // BLOCK, T % BLOCK
        for h in range(c["Hkv"]):
            k = (cache["k8"][b, h, :full].double() * cache["k_scale"][b, h, :full, None, None].double()).flatten(0, 1)
            v = (cache["v8"][b, h, :full].double() * cache["v_scale"][b, h, :full, None, None].double())
            k = torch.cat((k, cache["k_tail"][b, h, full % 2, :rest].double()))
            v = torch.cat((v.transpose(-1, -2).flatten(0, 1), cache["v_tail"][b, h, full % 2, :, :rest].double().T))
            for i in range(c["Lq"]):
                seen = start + i + 1
                w = torch.softmax(s["Q"][b, i, h * G:(h + 1) * G].double() @ k[:seen].T / math.sqrt(c["d"]), -1)
                o[b, i, h * G:(h + 1) * G] = w @ v[:seen]
    if c["gate"] != "none":
        sig = torch.sigmoid(s["X"].double() @ s["W_g"].double())
        o = o * (sig[..., None] if c["gate"] == "headwise" else sig.reshape(o.shape))
    return o
