"""What the token mixers are measured on: the 8-bit paged KV cache (written, read back), the attention of new tokens
over it, and the gated delta rule.  Each operator stands here in its plain form, in elementary torch operations in
fp32, beside the calls that a program makes of the library, with a 64-bit evaluation of its definition (`exact`)."""
import math
import random

import torch

own = False

DEV = "cuda"

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
#
# Head layouts: the model width 2560 as 20 heads of 128 or 10 of 256 (and neighbours), 64 for small models; the
# gated delta rule at 16 / 32 heads of 128.  New tokens per sequence: 1 (decode), 2-8 (verify windows), chunks of a
# prompt.  "lens" says how sequence lengths are spread: "same", or "ragged" (from a few tokens up to the largest).


def listed():
    return [
        # one verify window of four tokens enters the cache of one long sequence: latency
        dict(name="write verify window", op="write", fmt="int8", n_seqs=1, max_new=4, max_kv=4099, heads=20, kv_heads=4, dim=128, page=64, lens="same"),
        # the prompts of five requests enter the cache, ragged
        dict(name="write prompts", op="write", fmt="e4m3", n_seqs=5, max_new=8191, max_kv=8191, heads=10, kv_heads=2, dim=256, page=32, lens="ragged"),
        # a long prefix leaves the cache (moved to another replica)
        dict(name="read prefix", op="read", fmt="int8", n_seqs=1, max_new=32768, max_kv=32768, heads=20, kv_heads=4, dim=128, page=64, lens="same"),
        # short ragged contexts leave the cache
        dict(name="read ragged", op="read", fmt="e4m3", n_seqs=7, max_new=613, max_kv=613, heads=8, kv_heads=2, dim=64, page=16, lens="ragged"),
        # one user's next token: latency
        dict(name="decode one", op="attend", fmt="int8", n_seqs=1, max_new=1, max_kv=1023, heads=20, kv_heads=4, dim=128, page=64, causal=True, window=0, lens="same"),
        # a full batch of requests at ragged context lengths, one token each
        dict(name="decode batch", op="attend", fmt="int8", n_seqs=64, max_new=1, max_kv=16384, heads=20, kv_heads=4, dim=128, page=64, causal=True, window=0, lens="ragged"),
        # verify windows of four tokens over contexts up to 128K
        dict(name="verify long", op="attend", fmt="e4m3", n_seqs=8, max_new=4, max_kv=131072, heads=16, kv_heads=2, dim=256, page=128, causal=True, window=0, lens="ragged"),
        # a short prompt chunk per request in a sliding window, a key head per query head
        dict(name="window chunks", op="attend", fmt="e4m3", n_seqs=6, max_new=333, max_kv=5001, heads=8, kv_heads=8, dim=64, page=16, causal=True, window=1024, lens="ragged"),
        # a whole prompt of the prefill workload
        dict(name="prefill", op="attend", fmt="int8", n_seqs=1, max_new=4096, max_kv=4096, heads=20, kv_heads=4, dim=128, page=64, causal=True, window=0, lens="same"),
        # a chunk of a long prompt behind 30K tokens of context
        dict(name="chunk of long prompt", op="attend", fmt="int8", n_seqs=1, max_new=2048, max_kv=32768, heads=10, kv_heads=2, dim=256, page=64, causal=True, window=0, lens="same"),
        # verify windows through the recurrent state of sixteen requests
        dict(name="delta verify", op="delta", n_seqs=16, max_new=4, heads=32, qk_heads=16, dim_k=128, dim_v=128, l2norm=True, lens="same"),
        # ragged prompts through the chunked form
        dict(name="delta prompts", op="delta", n_seqs=3, max_new=4096, heads=32, qk_heads=16, dim_k=128, dim_v=128, l2norm=True, lens="ragged"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "delta", "delta"])
    if op == "delta":
        many = rng.random() < 0.5
        qk = rng.choice([2, 4, 8, 16])
        return dict(op=op, n_seqs=_log_int(rng, 1, 6 if many else 48), max_new=_log_int(rng, 33, 2500) if many else rng.randint(1, 8),
                    heads=qk * rng.choice([1, 2]), qk_heads=qk, dim_k=rng.choice([64, 128]), dim_v=rng.choice([64, 128]),
                    l2norm=rng.random() < 0.5, lens=rng.choice(["same", "ragged"]))
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    case = dict(op=op, fmt=rng.choice(["int8", "e4m3"]), kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 8]),
                dim=dim, page=rng.choice([16, 32, 64, 128, 256]), lens=rng.choice(["same", "ragged"]))
    if op != "attend":
        n_seqs = _log_int(rng, 1, 32)
        max_new = _log_int(rng, 1, max(2, 16384 // n_seqs))
        return dict(case, n_seqs=n_seqs, max_new=max_new, max_kv=max_new + (_log_int(rng, 1, 8192) if op == "write" else 0))
    if rng.random() < 0.5:    # decode and verify windows
        n_seqs = _log_int(rng, 1, 48)
        max_new = rng.randint(1, 8)
        max_kv = _log_int(rng, max_new, 16384 if n_seqs > 4 else 65536)
        if n_seqs * max_kv * kv_heads * dim > 1 << 28:
            max_kv = max(max_new, (1 << 28) // (n_seqs * kv_heads * dim))
    else:                     # chunks
        n_seqs = _log_int(rng, 1, 4)
        max_new = _log_int(rng, 9, 2048 // n_seqs)
        max_kv = max_new + _log_int(rng, 1, 8192)
    causal = rng.random() < 0.8
    return dict(case, n_seqs=n_seqs, max_new=max_new, max_kv=max_kv, causal=causal,
                window=_log_int(rng, 1, 4096) if causal and rng.random() < 0.3 else 0)


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence, fixed by the case."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, kv = [], []
    for s in range(case["n_seqs"]):
        n, m = case["max_new"], case.get("max_kv", 0)
        if case["lens"] == "ragged" and s > 0:    # the first sequence has the largest lengths
            if n > 8:
                n = rng.randint(1, n)
            m = n if case["op"] == "read" else n + int((m - n) * rng.random())
        new.append(n)
        kv.append(max(m, n))
    return new, kv


def _visible(case):
    """Keys that a sequence's new tokens read, and (query, key) pairs, summed over the sequences."""
    keys = pairs = 0
    for n, m in zip(*_lengths(case)):
        if not case["causal"]:
            keys, pairs = keys + m, pairs + n * m
            continue
        w = case["window"] or m + 1
        first = m - n                                  # position of the first new token
        keys += m - max(0, first + 1 - w)
        full = max(0, min(n, w - 1 - first))           # tokens whose window reaches position 0
        pairs += full * (first + 1) + full * (full - 1) // 2 + (n - full) * w
    return keys, pairs


def work(case):
    new, kv = _lengths(case)
    T = sum(new)
    if case["op"] == "delta":
        H, Hq, dk, dv = case["heads"], case["qk_heads"], case["dim_k"], case["dim_v"]
        return {"bytes": T * (2 * 2 * Hq * dk + 2 * 2 * H * dv + 8 * H) + case["n_seqs"] * 2 * 4 * H * dk * dv,
                "flops": 6 * T * H * dk * dv}
    row, scale = case["kv_heads"] * case["dim"], 4 * case["kv_heads"]
    if case["op"] == "write":      # the new rows in, codes and scales out, both back, the values out
        return {"bytes": 2 * T * (2 * row + 2 * (row + scale) + 2 * row), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * T * (row + scale + 2 * row), "flops": 0}
    keys, pairs = _visible(case)
    return {"bytes": 2 * keys * (row + scale) + T * case["heads"] * (4 * case["dim"] + 4),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _starts(new):
    t = torch.tensor([0] + new)
    return t.cumsum(0).to(torch.int32).to(DEV)


def _encode(x, fmt):
    """Rows of x in 8 bits: codes, and a scale per row."""
    x = x.float()
    a = x.abs().amax(-1)
    top = 127.0 if fmt == "int8" else 448.0
    safe = torch.where(a > 0, a, torch.ones_like(a))
    y = x * top / safe[..., None]
    codes = torch.round(y).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return codes, torch.where(a > 0, a / top, torch.ones_like(a))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    new, kv = _lengths(case)
    T, B = sum(new), case["n_seqs"]
    s = dict(case=case, q_start=_starts(new), n_tokens=T)
    if case["op"] == "delta":
        H, Hq, dk, dv = case["heads"], case["qk_heads"], case["dim_k"], case["dim_v"]
        q, k = normal(T, Hq, dk), normal(T, Hq, dk)
        if not case["l2norm"]:      # a program that normalises its queries and keys itself
            q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
        rate = torch.rand(H, generator=g, device=DEV) * 8 + 0.05
        s.update(q=q.bfloat16(), k=k.bfloat16(), v=normal(T, H, dv).bfloat16(),
                 log_decay=-rate * torch.nn.functional.softplus(normal(T, H) - 4.0), beta=torch.sigmoid(normal(T, H)),
                 states=torch.zeros(2 * B, H, dk, dv, device=DEV), scale=dk ** -0.5,
                 src=torch.arange(B, device=DEV, dtype=torch.int32), dst=torch.arange(B, 2 * B, device=DEV, dtype=torch.int32))
        s["states"][:B] = 0.3 * normal(B, H, dk, dv)
        return s
    Hk, d, page = case["kv_heads"], case["dim"], case["page"]
    per_seq = [-(-m // page) for m in kv]
    n_pages = sum(per_seq) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, max(per_seq), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(per_seq):
        table[i, :n] = order[at:at + n]
        at += n
    s.update(kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV), table=table, n_pages=n_pages)
    # what the pages hold: rows of unequal size, as layers' keys and values have
    for n in ("k", "v"):
        x = normal(n_pages, Hk, page, d) * torch.exp(0.5 * normal(n_pages, Hk, page, 1))
        s[n + "_codes"], s[n + "_scale"] = _encode(x, case["fmt"])
        del x
    if case["op"] == "write":
        # keys and values are slices of the fused projection's rows
        qkv = (normal(T, (case["heads"] + 2 * Hk) * d) * torch.exp(0.5 * normal(T, 1))).bfloat16()
        kv_cols = qkv[:, case["heads"] * d:].view(T, 2 * Hk, d)
        s.update(k=kv_cols[:, :Hk], v=kv_cols[:, Hk:])
    elif case["op"] == "attend":
        s.update(q=(1.5 * normal(T, case["heads"], d)).bfloat16(), scale=d ** -0.5)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------


def _token_rows(s):
    """Sequence, and position in the sequence's cache, of each new token."""
    t = torch.arange(s["n_tokens"], device=DEV)
    seq = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    last = s["q_start"].long()[seq + 1]
    return seq, s["kv_len"].long()[seq] - last + t


def _slots(s):
    seq, pos = _token_rows(s)
    page = s["case"]["page"]
    return s["table"][seq, pos // page].long(), pos % page


def _read_plain(s):
    pages, at = _slots(s)
    return tuple((s[n + "_codes"][pages, :, at].float() * s[n + "_scale"][pages, :, at][..., None]).bfloat16() for n in "kv")


def _write_plain(s):
    pages, at = _slots(s)
    for n in "kv":
        codes, scale = _encode(s[n], s["case"]["fmt"])
        # (8-bit floats are moved as bytes)
        s[n + "_codes"].view(torch.uint8)[pages, :, at] = codes.view(torch.uint8)
        s[n + "_scale"][pages, :, at] = scale
    return _read_plain(s)


def _padded(s):
    """[sequences, most new tokens] -> row of the packed tokens, and which of them exist."""
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(s["case"]["max_new"], device=DEV)
    there = i[None] < n[:, None]
    rows = s["q_start"][:-1].long()[:, None] + i[None]
    return torch.where(there, rows, 0), there, n


def _attend_plain(s):
    c = s["case"]
    Hk, d, B, N = c["kv_heads"], c["dim"], c["n_seqs"], c["max_new"]
    group = c["heads"] // Hk
    rows, there, n = _padded(s)
    L = s["table"].shape[1] * c["page"]

    def cached(name):      # [B, Hk, L, d]
        x = s[name + "_codes"].view(torch.uint8)[s["table"].long()].view(s[name + "_codes"].dtype).float()
        x *= s[name + "_scale"][s["table"].long()][..., None]
        return x.transpose(1, 2).reshape(B, Hk, L, d)

    q = s["q"].float()[rows].view(B, N, Hk, group, d).permute(0, 2, 1, 3, 4).reshape(B, Hk, N * group, d)
    x = (q @ cached("k").transpose(-1, -2)).mul_(s["scale"]).view(B, Hk, N, group, L)
    key = torch.arange(L, device=DEV)
    seen = (key < s["kv_len"].long()[:, None])[:, None]                                # [B, 1, L]
    if c["causal"]:
        pos = (s["kv_len"].long() - n)[:, None] + torch.arange(N, device=DEV)          # [B, N]
        seen = seen & (key <= pos[..., None])
        if c["window"]:
            seen = seen & (key > pos[..., None] - c["window"])
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hk, N * group, L) @ cached("v")).view(B, Hk, N, group, d) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hk * group, d), lse.permute(0, 2, 1, 3).reshape(B, N, Hk * group)
    return o[there].bfloat16(), lse[there]


def _delta_plain(s):
    c = s["case"]
    B, group = c["n_seqs"], c["heads"] // c["qk_heads"]
    rows, there, _ = _padded(s)
    q, k, v = (s[n].float() for n in "qkv")
    if c["l2norm"]:
        q, k = (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q, k = (x.repeat_interleave(group, 1)[rows] for x in (q * s["scale"], k))          # [B, N, H, dk]
    v = v[rows]
    decay = torch.where(there[..., None], s["log_decay"][rows], 0.0).exp()
    beta = torch.where(there[..., None], s["beta"][rows], 0.0)                         # a step past the end changes nothing
    S = s["states"][s["src"].long()]
    outs = []
    for t in range(c["max_new"]):      # the rule is a recurrence over the tokens
        S = S * decay[:, t, :, None, None]
        u = (v[:, t] - (k[:, t, :, None] @ S)[:, :, 0]) * beta[:, t, :, None]
        S = S + k[:, t, :, :, None] * u[:, :, None]
        outs.append((q[:, t, :, None] @ S)[:, :, 0])
    o = torch.stack(outs, 1)[there]
    s["states"][s["dst"].long()] = S
    return o.bfloat16(), s["states"][B:]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _handle(s):
    """The cache or the states, their batch description and workspace: what a program holds across its calls."""
    from latent_mixture_experts_softmax_b200 import mixers
    c, T, B = s["case"], s["n_tokens"], s["case"]["n_seqs"]
    if c["op"] == "delta":
        h = mixers.DeltaStates(c["heads"], c["qk_heads"], c["dim_k"], c["dim_v"], state=s["states"], l2norm=c["l2norm"])
        s["batch"] = h.batch(s["q_start"], s["src"], s["dst"], n_tokens=T, max_new=c["max_new"])
        s["ws"] = h.workspace(T, B, c["max_new"])
        s["out"] = torch.empty(T, c["heads"], c["dim_v"], dtype=torch.bfloat16, device=DEV)
    else:
        h = mixers.PagedKV(c["heads"], c["kv_heads"], c["dim"], c["page"], kv_fmt=c["fmt"],
                           buffers=(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]))
        s["batch"] = h.batch(s["q_start"], s["kv_len"], s["table"], n_tokens=T, max_new=c["max_new"])
        s["ws"] = h.workspace()
        if c["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(T, c["heads"], device=DEV)
        else:
            s["back"] = [torch.empty(T, c["kv_heads"], c["dim"], dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    s["handle"] = h
    return h


def run(s):
    c = s["case"]
    if not own:
        return {"write": _write_plain, "read": _read_plain, "attend": _attend_plain, "delta": _delta_plain}[c["op"]](s)
    h = s.get("handle") or _handle(s)
    if c["op"] == "delta":
        h.forward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["batch"], s["ws"], scale=s["scale"], out=s["out"])
        return s["out"], s["states"][c["n_seqs"]:]
    if c["op"] == "attend":
        h.attend(s["q"], s["batch"], s["ws"], scale=s["scale"], causal=c["causal"], window=c["window"], out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "write":
        h.append(s["k"], s["v"], s["batch"], s["ws"])
    return h.read(s["batch"], s["ws"], out=s["back"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _grid(y, fmt):
    """y on the grid of the codes, nearest, ties to even."""
    if fmt == "int8":
        return y.round()
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (y / step).round() * step


def _exact_cache(s, fmt):
    """[tokens, Hk, d] of each sequence's whole cache, keys and values, in fp64."""
    page = s["case"]["page"]
    got = []
    for i, m in enumerate(s["kv_len"].tolist()):
        at = torch.arange(m, device=DEV)
        pages = s["table"][i, at // page].long()
        got.append(tuple(s[n + "_codes"][pages, :, at % page].double() * s[n + "_scale"][pages, :, at % page].double()[..., None] for n in "kv"))
    return got


def _exact_attend(s):
    c = s["case"]
    group = c["heads"] // c["kv_heads"]
    starts = s["q_start"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for i, (K, V) in enumerate(_exact_cache(s, c["fmt"])):
        n, m = starts[i + 1] - starts[i], K.shape[0]
        pos = m - n + torch.arange(n, device=DEV)[:, None]
        j = torch.arange(m, device=DEV)[None]
        hidden = torch.zeros(n, m, dtype=torch.bool, device=DEV)
        if c["causal"]:
            hidden = j > pos
            if c["window"]:
                hidden |= j <= pos - c["window"]
        for h in range(c["heads"]):
            x = s["q"][starts[i]:starts[i + 1], h].double() @ K[:, h // group].T * s["scale"]
            x[hidden] = -math.inf
            some = ~hidden.all(1)
            z = torch.logsumexp(x, 1)
            w = torch.exp(x - z[:, None])
            out[starts[i]:starts[i + 1], h][some] = (w @ V[:, h // group])[some]
            lse[starts[i]:starts[i + 1], h] = z
    return out, lse


def _exact_delta(s, chunk=64):
    """In chunks: with the decays G from a chunk's start, U = (I + tril(b K K' G_i/G_j, -1))^-1 b (V - G K S)."""
    c = s["case"]
    group = c["heads"] // c["qk_heads"]
    q, k, v, g, b = (s[n].double().transpose(0, 1) for n in ("q", "k", "v", "log_decay", "beta"))
    if c["l2norm"]:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q, k = (x.repeat_interleave(group, 0) for x in (q * s["scale"], k))
    starts = s["q_start"].tolist()
    out = torch.empty(v.shape, dtype=torch.float64, device=DEV)
    states = s["states"][s["src"].long()].double()
    for i in range(c["n_seqs"]):
        S = states[i]
        for t in range(starts[i], starts[i + 1], chunk):
            w = slice(t, min(t + chunk, starts[i + 1]))
            G = g[:, w].cumsum(1)
            D = torch.exp(torch.tril(G[:, :, None] - G[:, None]))
            K, bb = k[:, w], b[:, w, None]
            A = torch.tril(bb * (K @ K.mT) * D, -1) + torch.eye(K.shape[1], dtype=torch.float64, device=DEV)
            U = torch.linalg.solve_triangular(A, bb * (v[:, w] - G.exp()[..., None] * (K @ S)), upper=False, unitriangular=True)
            out[:, w] = G.exp()[..., None] * (q[:, w] @ S) + torch.tril((q[:, w] @ K.mT) * D) @ U
            S = G[:, -1].exp()[:, None, None] * S + (K * (G[:, -1:] - G).exp()[..., None]).mT @ U
        states[i] = S
    return out.transpose(0, 1), states


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "delta":
        return _exact_delta(s)
    if case["op"] == "write":
        top = 127.0 if case["fmt"] == "int8" else 448.0
        got = []
        for n in "kv":
            x = s[n].double()
            a = x.abs().amax(-1, keepdim=True)
            a = torch.where(a == 0, 1.0, a)
            got.append(_grid(x * top / a, case["fmt"]) * a / top)
        return tuple(got)
    return tuple(torch.cat(x) for x in zip(*((K[K.shape[0] - n:], V[V.shape[0] - n:])
                                            for (K, V), n in zip(_exact_cache(s, case["fmt"]), _lengths(case)[0]))))
