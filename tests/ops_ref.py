"""Plain 64-bit implementations of the operators around the attention, for the
tests: per-head norm with rotary positions, the 8-bit cache, attention over it."""
import math

import numpy as np
import torch

BLOCK = 64


def half_step(dtype):
    """The most one rounding to ``dtype`` is off by, relative to the value."""
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------- norm and rotary positions
def frequencies(rd, theta=10000.0, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    w = []
    for i in range(rd // 2):
        base = theta * factor ** (rd / (rd - 2)) if scaling == "base" else theta
        f = base ** (-2.0 * i / rd)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            def index(turns):   # the pair that turns this often in orig_len positions
                return rd * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(theta))
            lo, hi = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rd - 1)
            u = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f / factor * u + f * (1 - u)
        w.append(f)
    return w


def norm_rope(x, gamma, positions, w, layout, scale=1.0, norm=True, eps=1e-6):
    """x [B, L, H, d] float64; positions [B, L]; w: frequencies (None: no rotation)."""
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if gamma is not None:
            x = x * gamma
    if w is None:
        return x
    rd = 2 * len(w)
    a = positions.double()[..., None, None] * torch.tensor(w, dtype=torch.float64, device=x.device)
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    r, rest = x[..., :rd], x[..., rd:]
    if layout == "half":
        u, v = r[..., :rd // 2], r[..., rd // 2:]
        return torch.cat((u * c - v * s, v * c + u * s, rest), -1)
    u, v = r[..., 0::2], r[..., 1::2]
    return torch.cat((torch.stack((u * c - v * s, v * c + u * s), -1).flatten(-2), rest), -1)


# ---------------------------------------------------------------- the 8-bit cache
def quantise(x, kind):
    """x [64, d] float64 of bf16 values -> (codes float64, scale float)."""
    amax = float(x.abs().max()) if not bool(torch.isnan(x).any()) else math.nan
    if amax == 0:
        return torch.zeros_like(x), 0.0
    if not math.isfinite(amax):
        return torch.zeros_like(x), math.nan
    if kind == "int8":
        scale = float(np.float32(amax) * (np.float32(1) / np.float32(127)))
        return torch.clamp(torch.round(x / scale), -127, 127), scale   # (torch.round: ties to even)
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    y = x / 2.0 ** e
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, 2.0 ** e


class RefCache:
    """One (sequence, head) of the cache: every token's K and V row in float64, and
    the blocks as they are held."""

    def __init__(self, kind, d):
        self.kind, self.d = kind, d
        self.k, self.v = torch.zeros(0, d, dtype=torch.float64), torch.zeros(0, d, dtype=torch.float64)

    def append(self, k, v):
        self.k, self.v = torch.cat((self.k, k.double().cpu())), torch.cat((self.v, v.double().cpu()))

    def held(self):
        """K and V as the attention sees them, [T, d] each."""
        out = []
        for x in (self.k, self.v):
            y = x.clone()
            for j in range(len(x) // BLOCK):
                q, s = quantise(x[j * BLOCK:(j + 1) * BLOCK], self.kind)
                y[j * BLOCK:(j + 1) * BLOCK] = q * s
            out.append(y)
        return out


def code_values(t):
    """The values of int8 or e4m3 codes, as float64 on the host."""
    return (t.cpu() if t.dtype == torch.int8 else t.cpu().float()).double()


def cache_rows(cache, b, h, T):
    """K and V [T, d] float64 of a Cache8 of T tokens, as its bytes say."""
    full, rest = T // BLOCK, T % BLOCK
    d = cache.d_k
    k = cache.k8[b, h, :full].float().double() * cache.k_scale[b, h, :full, None, None].double()
    v = cache.v8[b, h, :full].float().double() * cache.v_scale[b, h, :full, None, None].double()
    k = torch.cat((k.reshape(-1, d), cache.k_tail[b, h, full % 2, :rest].double()))
    v = torch.cat((v.transpose(-1, -2).reshape(-1, d), cache.v_tail[b, h, full % 2, :, :rest].double().T))
    return k, v


def attend(q, k, v, seen):
    """q [n, d], k, v [T, d] float64; row r sees the first seen[r] tokens. Returns the
    outputs, the weighted sum of |v| and, for the error bound of the scores, the
    largest sum of |q_c k_c| / sqrt(d) over the tokens seen."""
    d = q.shape[1]
    out, mag, top = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(len(q), dtype=torch.float64)
    for r in range(len(q)):
        n = int(seen[r])
        if n == 0:
            continue
        p = torch.softmax(q[r] @ k[:n].T / math.sqrt(d), -1)
        out[r], mag[r] = p @ v[:n], p @ v[:n].abs()
        top[r] = (q[r].abs() @ k[:n].abs().T).max() / math.sqrt(d)
    return out, mag, top
