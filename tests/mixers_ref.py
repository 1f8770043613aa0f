"""Plain 64-bit forms of the token mixers, sequence by sequence and row by row,
for the tests: written from the definitions in include/lmoe.h, on the CPU.

Every form gives the value and a bound of what the kernels' documented
roundings may move it by; u(t) is half a step of type t."""
import math

import numpy as np
import torch

U_BF16, U_FP16, U_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
TOP = {"int8": 127.0, "e4m3": 448.0}


def encode(x, fmt):
    """Codes (as values) and scales of bf16 rows, in exact arithmetic (fp64 quotients of 15-bit by 8-bit numbers)."""
    x = x.double()
    a = x.abs().amax(-1)
    tiny = a < 2.0 ** -100
    y = x * TOP[fmt] / torch.where(tiny, 1.0, a)[..., None]
    if fmt == "int8":
        c = y.round()
    else:
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        c = (y / step).round() * step
    bad = ~torch.isfinite(a)
    scale = (a.float() / TOP[fmt])                      # one fp32 division
    scale = torch.where(tiny, 1.0, torch.where(bad, math.nan, scale))
    c = torch.where((tiny | bad)[..., None], 0.0, c)
    return c, scale


class Cache:
    """A paged cache on the CPU: codes as fp32 values, scales, and a table of shuffled pages."""

    def __init__(self, fmt, Hk, D, page, kv, seed=0, spare=2, garbage=True):
        g = torch.Generator().manual_seed(seed)
        per = [-(-m // page) for m in kv]
        n = sum(per) + spare
        order = torch.randperm(n, generator=g).tolist()
        self.fmt, self.page, self.kv, self.n_pages = fmt, page, kv, n
        self.table = torch.full((len(kv), max(1, max(per))), -7, dtype=torch.int32)    # entries past the length are not read
        for s, m in enumerate(per):
            self.table[s, :m] = torch.tensor([order.pop() for _ in range(m)], dtype=torch.int32)
        self.codes, self.scale = {}, {}
        for name in "kv":
            if garbage:    # every place nobody wrote holds a NaN code and a NaN scale
                c = torch.full((n, Hk, page, D), math.nan if fmt == "e4m3" else -128.0)
                s = torch.full((n, Hk, page), math.nan)
            else:
                c, s = torch.zeros(n, Hk, page, D), torch.ones(n, Hk, page)
            self.codes[name], self.scale[name] = c, s
        for s, m in enumerate(kv):
            for name in "kv":
                x = (torch.randn(m, Hk, D, generator=g) * torch.exp(torch.randn(m, Hk, 1, generator=g))).bfloat16()
                self.put(name, s, range(m), x)

    def put(self, name, s, positions, x):
        c, sc = encode(x, self.fmt)
        for i, pos in enumerate(positions):
            at = self.table[s, pos // self.page].item()
            self.codes[name][at, :, pos % self.page] = c[i].float()
            self.scale[name][at, :, pos % self.page] = sc[i]

    def buffers(self, device):
        dt = torch.int8 if self.fmt == "int8" else torch.float8_e4m3fn
        return tuple(self.codes[n].to(dt).to(device) for n in "kv") + tuple(self.scale[n].to(device) for n in "kv")

    def rows(self, name, s, m=None):
        """[m, Hk, D] in fp64: the cached rows of a sequence."""
        m = self.kv[s] if m is None else m
        pos = torch.arange(m)
        at = self.table[s, pos // self.page].long()
        return self.codes[name][at, :, pos % self.page].double() * self.scale[name][at, :, pos % self.page].double()[..., None]


def attend(q, K, V, first, scale, causal, window):
    """One sequence: q [n, Hq, D] bf16 at positions first.., K, V [m, Hk, D] fp64.
    (out, lse, bound of out, bound of lse)."""
    n, Hq, D = q.shape
    m, Hk = K.shape[:2]
    q = q.double()
    pos, j = first + torch.arange(n)[:, None], torch.arange(m)[None]
    seen = torch.ones(n, m, dtype=torch.bool)
    if causal:
        seen = j <= pos
        if window:
            seen &= j > pos - window
    out, tol = torch.zeros(n, Hq, D, dtype=torch.float64), torch.zeros(n, Hq, D, dtype=torch.float64)
    lse, ltol = torch.full((n, Hq), -math.inf, dtype=torch.float64), torch.zeros(n, Hq, dtype=torch.float64)
    some = seen.any(1)
    for h in range(Hq):
        k, v = K[:, h * Hk // Hq], V[:, h * Hk // Hq]
        x = (q[:, h] @ k.T * scale).masked_fill(~seen, -math.inf)
        if not some.any():
            continue
        z = torch.logsumexp(x, 1)
        w = torch.exp(x - z[:, None])
        w[~some] = 0.0
        vv = torch.where(seen.any(0)[:, None], v, 0.0)       # a key nobody sees may hold anything
        w = torch.where(seen, w, 0.0)
        out[:, h] = w @ vv
        lse[:, h] = z
        # scores: D exact products summed in fp32 in any order (2 steps a sum, for a truncating adder), scaled, and
        # taken from the running maximum: four roundings of numbers up to the largest score
        ab = (q[:, h].abs() @ torch.where(seen.any(0)[:, None], k, 0.0).abs().T * abs(scale)).masked_fill(~seen, 0.0).amax(1)
        ds = 2 * (D + 8) * U_F32 * ab + 8 * U_F32 * (ab + 40)
        # probabilities: 2^x to 2^-22, fp16 by half a step; sums over the keys in fp32
        dp = 2 * ds + 2.0 ** -21 + 2 * (m + 8) * U_F32
        mag = w @ vv.abs()
        out_err = (U_FP16 + 2 * dp)[:, None] * mag + 2.0 ** -24 * vv.abs().amax()    # p under fp16's smallest normal: half its step
        tol[:, h] = U_BF16 * (out[:, h].abs() + out_err) + out_err
        ltol[:, h] = dp + ds + 4 * U_F32 * z.abs().clamp_min(1.0)
    return out, lse, tol, ltol


def delta(q, k, v, log_decay, beta, S, scale, l2norm):
    """The recurrence in fp64 over one sequence: q, k [n, Hq, DK], v [n, H, DV], S [H, DK, DV] -> (out, S)."""
    n, H = log_decay.shape
    group = H // q.shape[1]
    q, k, v, b = q.double(), k.double(), v.double(), beta.double()
    a = torch.exp(log_decay.double())
    if l2norm:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q, k = (x.repeat_interleave(group, 1) for x in (q * scale, k))
    S = S.double().clone()
    out = torch.zeros(n, H, v.shape[-1], dtype=torch.float64)
    for t in range(n):
        S = S * a[t, :, None, None]
        u = (v[t] - torch.einsum("hk,hkv->hv", k[t], S)) * b[t, :, None]
        S = S + k[t, :, :, None] * u[:, None]
        out[t] = torch.einsum("hk,hkv->hv", q[t], S)
    return out, S


def assert_within(got, want, tol, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN where none is due, or none where one is"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    fine = ~torch.isnan(want) & ~inf
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: off by {(got - want).abs()[fine].max():.3e}, {over.max():.3e} more than its bound"


def starts(ns):
    return torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32)
