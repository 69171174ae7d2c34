"""Plain implementations of the paged 4-bit cache for the tests, from the header's
formulas: the plan of a step, a page's bytes, codes and scales, and the attention's
error bound."""
import math

import numpy as np
import torch

from ops_ref import half_step

PAGE, GROUP = 64, 16
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
CODES = {"int4": [float(c - 8) for c in range(16)], "e2m1": E2M1 + [-x for x in E2M1]}
TOP = {"int4": 7.0, "e2m1": 6.0}
SCALES = [math.nan if b % 128 == 127 else (-1.0 if b > 127 else 1.0) * (b % 8 / 8 * 2.0 ** -6 if b % 128 < 8 else
          (1 + b % 8 / 8) * 2.0 ** (b % 128 // 8 - 7)) for b in range(256)]


def pages_of(tokens):
    return -(-tokens // PAGE)


# ---------------------------------------------------------------- the plan of a step
def plan(lens, new, table, free, n_free, n_rows, width, keep=None):
    """Lists in, lists out: cu, granted, slots, positions, what is free, and table and stack as
    they are after. For numbers in range."""
    keep = lens if keep is None else keep
    table, stack = [list(r) for r in table], list(free[:n_free])
    for b, (held, kept) in enumerate(zip(lens, keep)):
        stack += table[b][pages_of(kept):pages_of(held)]
    top, asked, left = len(stack), 0, len(stack)
    cu, granted, slots, positions = [0], [], [], []
    for b, (kept, n) in enumerate(zip(keep, new)):
        need = pages_of(kept + n) - pages_of(kept)
        asked += need
        ok = need == 0 or asked <= top
        for k in range(need if ok else 0):
            left -= 1
            table[b][pages_of(kept) + k] = stack[left]
        granted.append(n if ok else 0)
        cu.append(cu[-1] + n)
        for p in range(kept, kept + n):
            positions.append(p)
            slots.append(table[b][p // PAGE] * PAGE + p % PAGE if ok else -1)
    rest = n_rows - len(slots)
    return cu, granted, slots + [-1] * rest, positions + [0] * rest, left, table, stack


# ---------------------------------------------------------------- a page's bytes
def places(d, kind):
    """Byte and shift of every key code and value code [64, d, 2], byte of every key and value scale
    [64, d / 16], in the 72 d bytes of a page's head."""
    n, c = np.meshgrid(np.arange(PAGE), np.arange(d), indexing="ij")
    j, r = c // 16, c % 16
    t, p, s = r // 4, r // 2 % 2, r % 2
    start = n * d // 2 + t * d // 8
    if kind == "e2m1":
        k = np.stack((start + 2 * j + p, 4 * s), -1)
    else:
        bit = 16 * s + 4 * (2 * (j % 2) + p)
        k = np.stack((start + 4 * (j // 2) + bit // 8, bit % 8), -1)
    g, high, tt = r % 8, r // 8, n % 8 // 2
    token = 2 * (n % 16 // 8) + n % 2                       # among 2 t, 2 t + 1, 2 t + 8, 2 t + 9
    byte = token if kind == "e2m1" else np.array([0, 2, 1, 3])[token]
    word = (((n // 16) * (d // 64) + j // 4) * 8 + g) * 16 + tt * 4 + j % 4
    v = np.stack((36 * d + 4 * word + byte, 4 * high), -1)
    n, j = np.meshgrid(np.arange(PAGE), np.arange(d // 16), indexing="ij")
    ks = 32 * d + n * (d // 16) + j
    vs = 68 * d + 4 * ((n // 16 * 4 + n % 8 // 2) * (d // 16) + j) + 2 * (n % 16 // 8) + n % 2
    return [torch.from_numpy(x) for x in (k, v, ks, vs)]


def codes_and_scales(pool, slots, kind):
    """Of tokens at slots: codes' values k, v [n, H, d] and scales ks, vs [n, H, d / 16] (without 2^exp), float64."""
    d, H, dev = pool.shape[2] // 72, pool.shape[1], pool.device
    k, v, ks, vs = (x.to(dev) for x in places(d, kind))
    slots = torch.as_tensor(slots, device=dev, dtype=torch.int64)
    page, at = slots // PAGE, slots % PAGE
    base = ((page[:, None] * H + torch.arange(H, device=dev)) * (72 * d))[..., None]      # [n, H, 1]
    flat = pool.reshape(-1)
    table = torch.tensor(CODES[kind], dtype=torch.float64, device=dev)
    scale = torch.tensor(SCALES, dtype=torch.float64, device=dev)

    def codes(where):
        w = where[at][:, None]
        return table[flat[base + w[..., 0]].long() >> w[..., 1] & 15]

    return codes(k), codes(v), scale[flat[base + ks[at][:, None]].long()], scale[flat[base + vs[at][:, None]].long()]


def held(cache, slots):
    """Keys and values at slots as the cache's bytes say, float64 [n, H, d]."""
    k, v, ks, vs = codes_and_scales(cache.pool, slots, cache.kind)
    return (k * ks.repeat_interleave(GROUP, -1) * 2.0 ** cache.k_exp, v * vs.repeat_interleave(GROUP, -1) * 2.0 ** cache.v_exp)


def quantise(x, kind, exp):
    """x [..., d] float64 of bf16 values, on the host -> codes' values [..., d] and scales [..., d / 16] float64."""
    x = x.unflatten(-1, (-1, GROUP))
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    down = (amax * 2.0 ** -exp).float().numpy()
    want = torch.from_numpy(down * (np.float32(1) / np.float32(TOP[kind]))).double().nan_to_num(0.0, 3e38).clamp(max=448.0)
    grid = torch.tensor(SCALES[:127], dtype=torch.float64)
    up = torch.searchsorted(grid, want.contiguous()).clamp(max=126)
    low = (up - 1).clamp(min=0)
    a, b = grid[up] - want, want - grid[low]
    byte = torch.where((a < b) | ((a == b) & (up % 2 == 0)), up, low)
    scale = torch.where(bad, 0.0, grid[byte])
    y = torch.where(scale[..., None] > 0, x / (scale[..., None] * 2.0 ** exp), torch.zeros_like(x))
    y = torch.where(bad[..., None], torch.zeros_like(y), y).clamp(-TOP[kind], TOP[kind])
    if kind == "int4":
        codes = torch.round(y)
    else:
        mag = torch.tensor(E2M1, dtype=torch.float64)
        off = (y.abs()[..., None] - mag).abs()
        # of two equally near the even one (nearest to 2 i, i. e. a hair less off)
        near = off - 1e-9 * (torch.arange(8) % 2 == 0)
        codes = mag[near.argmin(-1)] * torch.sign(y)
    return codes.flatten(-2), torch.where(bad, math.nan, scale)


# ---------------------------------------------------------------- the attention, to the kernel's bound
def check_attention(O, X, Q, cache, table, lens, new, cu, W, gate, requests=None, more=16.0):
    """Every row against the formula in 64 bits, on the cache's own bytes. With A the sum of weights times |v|:
    a score's 16-column sums are those of exact products, in float32, and so is their sum over the groups: d additions of
    2^-23 of the sum of |q_c| (|code| + more) scale; more, of int4 alone, is room for a kernel that sums codes + 8 and
    takes 8 off: 0 where the codes are summed. A weight is rounded to fp16 twice, 2^-11 each, and nothing is finer than 2^-38 W (see the header). The sums of
    weights and values are float32 too, over T / 16 products of 16 tokens (with more as many again), 2^-23 of the running
    sum each; 2^-16 covers the exponentials (2 ulp of an argument below 2^7 in magnitude), sums of weights and the
    gate's sigmoid. Then the output is rounded to bf16."""
    d, H = cache.d_k, cache.H_kv
    Hq = Q.shape[1]
    G = Hq // H
    more = more if cache.kind == "int4" else 0.0
    done = torch.zeros(len(Q), dtype=torch.bool, device=Q.device)
    for b in range(len(lens)) if requests is None else requests:
        n, T, at = new[b], lens[b] + new[b], cu[b]
        done[at:at + n] = True
        if n == 0:
            continue
        pos = torch.arange(T, device=Q.device)
        slots = table[b].to(Q.device).long()[pos // PAGE] * PAGE + pos % PAGE
        kc, vc, ks, vs = codes_and_scales(cache.pool, slots, cache.kind)
        ks = ks.repeat_interleave(GROUP, -1) * 2.0 ** cache.k_exp
        up = 2.0 ** cache.v_exp
        wide = vs.repeat_interleave(GROUP, -1)
        k, km, v, vm, unit = (x.transpose(0, 1) for x in (kc * ks, (kc.abs() + more) * ks, vc * wide * up,
                                                           (vc.abs() + more) * wide * up, vc.abs() * (1 + wide) * up))
        q = Q[at:at + n].double().view(n, H, G, d).permute(1, 0, 2, 3).reshape(H, n * G, d)
        seen = pos <= lens[b] + torch.arange(n, device=Q.device).repeat_interleave(G)[:, None]
        w = torch.softmax((q @ k.transpose(1, 2) / math.sqrt(d)).masked_fill(~seen, -math.inf), -1)
        top = (q.abs() @ km.transpose(1, 2)).masked_fill(~seen, 0).amax(-1, keepdim=True) / math.sqrt(d)
        ref, A, Am = w @ v, w @ v.abs(), w @ vm
        page_top = torch.stack([c.amax((0, 2)) for c in vs.split(PAGE)], -1)               # [H, pages]
        page_top = torch.exp2(torch.ceil(torch.log2(page_top.clamp(min=1.0) * 1.0000001)))
        largest = (w * page_top.repeat_interleave(PAGE, -1)[:, None, :T]).amax(-1, keepdim=True)
        tol = (2 * half_step(torch.float16) + 2 * d * 2.0 ** -23 * top + 2.0 ** -16) * A
        tol = tol + (T / (4 if more else 8) + 32) * 2.0 ** -23 * Am + 2.0 ** -38 * largest * (seen.double() @ unit)
        sig = torch.ones(n, Hq, d, dtype=torch.float64, device=Q.device)
        if gate != "none":
            s = torch.sigmoid(X[at:at + n].double() @ W.double())
            sig = s[..., None].expand(-1, -1, d) if gate == "headwise" else s.view(n, Hq, d)

        def rows(t):
            return t.view(H, n, G, d).permute(1, 0, 2, 3).reshape(n, Hq, d) * sig
        ref, tol = rows(ref), rows(tol) + half_step(torch.bfloat16) * rows(ref).abs() + 1e-30
        err = (O[at:at + n].double() - ref).abs()
        assert bool((err <= tol).all()), (b, T, float((err / tol).max()))
    if requests is None:
        assert not bool(O[~done].any()), "rows that count for no request are not zero"
