"""The token mixers on the GPU against their 64-bit forms (tests/mixers_ref.py)."""
import math

import pytest
import torch

from latent_mixture_experts_softmax_b200 import binding as B
from latent_mixture_experts_softmax_b200 import build, mixers

import mixers_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_all()
    assert torch.cuda.is_available()


def paged(cache, Hq, Hk, D):
    return mixers.PagedKV(Hq, Hk, D, cache.page, kv_fmt=cache.fmt, buffers=cache.buffers(DEV))


def batch_of(kv, cache, ns, pad=0, max_new=None, lens=None):
    return kv.batch(R.starts(ns).to(DEV), torch.tensor(cache.kv if lens is None else lens, dtype=torch.int32, device=DEV), cache.table.to(DEV),
                    n_tokens=sum(ns) + pad, max_new=max(ns) if max_new is None else max_new)


# ----------------------------------------------------------------------------
# the cache
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,Hk,page,ns,kv", [
    (64, 1, 16, [1], [1]),
    (64, 3, 32, [5, 0, 17], [40, 9, 17]),
    (128, 2, 16, [33, 1, 70], [33, 1000, 75]),
    (256, 1, 64, [130, 2], [131, 2]),
    (128, 5, 1024, [3], [2000]),
    (128, 2, 16, [9, 4], [5, 0]),          # fewer places than new tokens
])
def test_append_and_read(fmt, D, Hk, page, ns, kv):
    cache = R.Cache(fmt, Hk, D, page, kv, seed=D + Hk)
    pk = paged(cache, Hk, Hk, D)
    ws = pk.workspace()
    T, pad = sum(ns), 3
    g = torch.Generator().manual_seed(1)
    # slices of wider rows, as a fused projection leaves them
    wide = (torch.randn(T + pad, 2 * Hk + 1, D, generator=g) * torch.exp(2 * torch.randn(T + pad, 2 * Hk + 1, 1, generator=g))).bfloat16()
    wide[0, 0, :8] = torch.tensor([1.0, 0.5, -0.5, 0.25, 1.0, -1.0, 0.75, 0.0]) * wide[0, 0].abs().max()   # ties at 63.5
    k, v = wide[:, :Hk], wide[:, Hk:2 * Hk]
    dk = wide.to(DEV)
    b = batch_of(pk, cache, ns, pad)
    before = [t.clone() for t in (pk.k.view(torch.uint8), pk.v.view(torch.uint8), pk.k_scale, pk.v_scale)]
    pk.append(dk[:, :Hk], dk[:, Hk:2 * Hk], b, ws)
    t0 = 0
    for s, n in enumerate(ns):
        new = [(i, kv[s] - n + i) for i in range(n) if kv[s] - n + i >= 0]
        for name, x in (("k", k), ("v", v)):
            cache.put(name, s, [p for _, p in new], x[[t0 + i for i, _ in new]])
        t0 += n
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK
    # every place of the cache, those that nothing was written to included, bit for bit
    for got, want in zip((pk.k, pk.v, pk.k_scale, pk.v_scale), cache.buffers("cpu")):
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
    del before
    out = [torch.full((T + pad, Hk, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    pk.read(b, ws, out=out)
    t0 = 0
    for s, n in enumerate(ns):
        for name, o in zip("kv", out):
            want = torch.zeros(n, Hk, D, dtype=torch.float64)
            some = max(0, n - kv[s])
            if n > some:
                want[some:] = cache.rows(name, s)[kv[s] - n + some:]
            R.assert_within(o[t0:t0 + n], want, R.U_BF16 * want.abs() * (1 + 2 * R.U_F32) + 2 * R.U_F32 * want.abs(), f"read {name} of sequence {s}")
        t0 += n
    for o in out:
        assert (o[T:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_of_rows_at_the_ends_of_the_range(fmt):
    """Zero rows, tiny and huge rows, rows with an infinity or a NaN; the neighbours of a bad row are not touched by it."""
    D, page = 128, 16
    x = torch.randn(10, 1, D).bfloat16()
    x[0] = 0
    x[1] *= 2.0 ** -110
    x[2] *= 2.0 ** -90
    x[3] = (x[3].float() * 2.0 ** 120).bfloat16()
    x[4, 0, 5] = math.inf
    x[6, 0, 7] = math.nan
    x[8, 0, :] = torch.finfo(torch.bfloat16).max
    cache = R.Cache(fmt, 1, D, page, [10])
    pk = paged(cache, 1, 1, D)
    ws = pk.workspace()
    b = batch_of(pk, cache, [10])
    pk.append(x.to(DEV), x.to(DEV), b, ws)
    assert B.lmoe_last_device_status(ws) == B.LMOE_ERR_DEVICE_CHECK
    cache.put("k", 0, range(10), x)
    page0 = cache.table[0, 0].item()
    want_c, want_s = cache.codes["k"][page0, 0, :10], cache.scale["k"][page0, 0, :10]
    assert torch.equal(pk.k[page0, 0, :10].float().cpu(), want_c)
    assert torch.equal(pk.k_scale[page0, 0, :10].cpu().nan_to_num(-1), want_s.nan_to_num(-1))
    q = torch.randn(10, 1, D).bfloat16()
    out = pk.attend(q.to(DEV), b, ws).float().cpu()
    assert torch.isfinite(out[:3]).all() and torch.isnan(out[4:]).all()      # causal: rows 4 and later see the bad key


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------

def check_attend(fmt, Hq, Hk, D, page, ns, kv, causal=True, window=0, seed=0, pad=0, qmul=1.0, max_new=None, scale=None):
    cache = R.Cache(fmt, Hk, D, page, kv, seed=seed)
    pk = paged(cache, Hq, Hk, D)
    ws = pk.workspace()
    T = sum(ns)
    g = torch.Generator().manual_seed(seed + 1)
    wide = (torch.randn(T + pad, Hq + 1, D, generator=g) * qmul).bfloat16()
    q = wide[:, :Hq]
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((T + pad, Hq, D), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + pad, Hq), 5.0, device=DEV)
    b = batch_of(pk, cache, ns, pad, max_new)
    pk.attend(wide.to(DEV)[:, :Hq], b, ws, scale=scale, causal=causal, window=window, out=out, lse=lse)
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK
    t0 = 0
    for s, n in enumerate(ns):
        want, wl, tol, ltol = R.attend(q[t0:t0 + n], cache.rows("k", s), cache.rows("v", s), kv[s] - n, scale, causal, window)
        R.assert_within(out[t0:t0 + n], want, tol, f"out of sequence {s}")
        R.assert_within(lse[t0:t0 + n], wl, ltol, f"lse of sequence {s}")
        t0 += n
    assert (out[T:] == 5.0).all() and (lse[T:] == 5.0).all()
    first = out.clone(), lse.clone()
    pk.attend(wide.to(DEV)[:, :Hq], b, ws, scale=scale, causal=causal, window=window, out=out, lse=lse)
    assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse.nan_to_num(9), first[1].nan_to_num(9))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hk,D,page,ns,kv", [
    (1, 1, 64, 16, [1], [1]),
    (4, 2, 128, 16, [1], [15]),
    (20, 4, 128, 64, [1, 1, 1], [1023, 1, 129]),
    (20, 4, 128, 64, [4, 1, 3, 0], [300, 16, 3, 50]),
    (16, 2, 256, 32, [1, 1], [700, 33]),              # 8 rows
    (10, 1, 256, 128, [1], [513]),                    # 16 rows
    (16, 2, 256, 64, [4, 4], [1000, 70]),             # 32 rows
    (7, 7, 64, 16, [8, 2, 5], [90, 300, 5]),
    (12, 4, 64, 256, [5], [1500]),                    # 15 rows of 16
    (6, 2, 128, 16, [8], [40]),                       # 24 rows of 32
    (36, 1, 128, 16, [1], [200]),                     # more rows than one tile
])
def test_attend_few_tokens(fmt, Hq, Hk, D, page, ns, kv):
    check_attend(fmt, Hq, Hk, D, page, ns, kv, seed=Hq + D)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hk,D,page,ns,kv", [
    (4, 2, 64, 16, [70, 1, 33], [70, 200, 100]),
    (20, 4, 128, 64, [97], [400]),
    (8, 8, 128, 16, [257, 0, 130], [257, 10, 1000]),
    (10, 2, 256, 32, [150, 2], [300, 513]),
    (5, 1, 256, 64, [129], [129]),
    (64, 1, 64, 16, [6, 3], [6, 77]),
])
def test_attend_chunks(fmt, Hq, Hk, D, page, ns, kv):
    check_attend(fmt, Hq, Hk, D, page, ns, kv, seed=Hq + D, pad=2)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 70), (False, 0)])
@pytest.mark.parametrize("Hq,Hk,D,page,ns,kv", [
    (8, 1, 64, 16, [140, 1], [700, 70]),
    (10, 2, 128, 64, [210, 0, 30], [210, 9, 400]),
    (5, 1, 256, 128, [110, 3], [300, 65]),
])
def test_attend_many_row_tiles(fmt, causal, window, Hq, Hk, D, page, ns, kv):
    """More than four row tiles per key head."""
    check_attend(fmt, Hq, Hk, D, page, ns, kv, causal=causal, window=window, seed=Hq + D, pad=1)


@pytest.mark.parametrize("pages,kv_heads", [(1200, 3), (2000, 3), (3000, 2), (6000, 2)])
def test_attend_with_room_for_long_contexts(pages, kv_heads):
    """Page tables so wide that a launch takes several sequences, one, some heads of one, or none as images."""
    D, page, ns, kv = 256, 16, [90, 91, 2], [100, 150, 40]
    cache = R.Cache("int8", kv_heads, D, page, kv, seed=pages)
    cache.table = torch.cat([cache.table, torch.full((3, pages - cache.table.shape[1]), -7, dtype=torch.int32)], 1)
    pk = paged(cache, 6 * kv_heads, kv_heads, D)
    ws = pk.workspace()
    q = torch.randn(sum(ns), 6 * kv_heads, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    out = pk.attend(q.to(DEV), batch_of(pk, cache, ns), ws)
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK
    t0 = 0
    for s, n in enumerate(ns):
        want, _, tol, _ = R.attend(q[t0:t0 + n], cache.rows("k", s), cache.rows("v", s), kv[s] - n, D ** -0.5, True, 0)
        R.assert_within(out[t0:t0 + n], want, tol, f"out of sequence {s}")
        t0 += n


@pytest.mark.parametrize("window", [1, 16, 100])
@pytest.mark.parametrize("Hq,Hk,D,ns,kv", [(4, 2, 128, [1, 3], [500, 40]), (4, 4, 64, [200, 5], [301, 5]), (4, 2, 256, [40], [150])])
def test_attend_window(window, Hq, Hk, D, ns, kv):
    check_attend("int8", Hq, Hk, D, 16, ns, kv, window=window, seed=window)


@pytest.mark.parametrize("Hq,Hk,D,ns,kv", [(4, 2, 128, [1, 3], [500, 40]), (4, 4, 64, [100, 5], [301, 2]), (6, 2, 256, [70], [333])])
def test_attend_without_a_causal_mask(Hq, Hk, D, ns, kv):
    check_attend("e4m3", Hq, Hk, D, 32, ns, kv, causal=False, seed=D)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_without_a_key_are_zeros(D):
    """Fewer cached tokens than new ones (negative positions), an empty cache, padding rows behind the last sequence."""
    check_attend("int8", 4, 2, D, 16, [6, 3, 2], [4, 0, 2], pad=3)
    check_attend("e4m3", 4, 2, D, 16, [150, 40], [100, 0], pad=1)
    check_attend("e4m3", 4, 2, D, 16, [150, 40], [100, 0], causal=False)


@pytest.mark.parametrize("qmul,scale", [(1e-30, 1e30), (1e20, 1e-21), (30.0, None), (1.0, -0.2), (1.0, 0.0)])
def test_attend_scales(qmul, scale):
    check_attend("int8", 4, 2, 128, 16, [2], [100], qmul=qmul, scale=scale)
    check_attend("int8", 4, 2, 128, 16, [90], [100], qmul=qmul, scale=scale)


def test_value_rows_of_very_unequal_size():
    """A value's scale enters the exponent: rows 2^60 apart neither overflow nor vanish where they count."""
    for n in (1, 80):
        cache = R.Cache("int8", 1, 64, 16, [100])
        x = torch.randn(100, 1, 64) * torch.exp2(torch.linspace(-60, 60, 100))[torch.randperm(100)][:, None, None]
        cache.put("v", 0, range(100), x.bfloat16())
        pk = paged(cache, 2, 1, 64)
        ws = pk.workspace()
        q = torch.randn(n, 2, 64).bfloat16()
        out = pk.attend(q.to(DEV), batch_of(pk, cache, [n]), ws)
        want, _, tol, _ = R.attend(q, cache.rows("k", 0), cache.rows("v", 0), 100 - n, 0.125, True, 0)
        R.assert_within(out, want, tol, "out")


def test_a_nan_key_reaches_only_the_queries_that_see_it():
    for n in (5, 100):
        cache = R.Cache("int8", 1, 128, 16, [200])
        x = torch.randn(1, 1, 128).bfloat16()
        x[0, 0, 3] = math.nan
        bad = 200 - n // 2
        cache.put("k", 0, [bad], x)
        cache.put("v", 0, [bad], x)
        pk = paged(cache, 2, 1, 128)
        ws = pk.workspace()
        q = torch.randn(n, 2, 128).bfloat16()
        out = pk.attend(q.to(DEV), batch_of(pk, cache, [n]), ws).float().cpu()
        at = bad - (200 - n)
        assert torch.isfinite(out[:at]).all() and torch.isnan(out[at:]).all()


def test_a_nan_query_is_alone():
    for n in (3, 50):
        cache = R.Cache("e4m3", 1, 64, 16, [64])
        pk = paged(cache, 4, 1, 64)
        ws = pk.workspace()
        q = torch.randn(n, 4, 64).bfloat16()
        q[1, 2, 9] = math.nan
        q[2, 0, 1] = -math.inf
        out = pk.attend(q.to(DEV), batch_of(pk, cache, [n]), ws).float().cpu()
        nan = torch.isnan(out).all(-1)
        assert nan[1, 2] and nan[2, 0] and nan.sum() == 2 and not torch.isnan(out[~nan]).any()


# ----------------------------------------------------------------------------
# bad batches (after the kernels' checks have been read on the CPU: every
# index is compared before it is used)
# ----------------------------------------------------------------------------

def test_bad_pages_are_reported_and_masked():
    for n in (2, 90):
        cache = R.Cache("int8", 2, 64, 16, [100, 100])
        pk = paged(cache, 4, 2, 64)
        ws = pk.workspace()
        table = cache.table.clone()
        table[0, 0], table[0, 1] = cache.n_pages, -1
        q = torch.randn(2 * n, 4, 64).bfloat16()
        b = pk.batch(R.starts([n, n]).to(DEV), torch.tensor([100, 100], dtype=torch.int32, device=DEV), table.to(DEV), 2 * n, n)
        out = pk.attend(q.to(DEV), b, ws)
        assert B.lmoe_last_device_status(ws) == B.LMOE_ERR_DEVICE_CHECK
        K, V = cache.rows("k", 0), cache.rows("v", 0)
        want, _, tol, _ = R.attend(q[:n], K[32:], V[32:], 100 - n - 32, 0.125, True, 0)
        R.assert_within(out[:n], want, tol, "the sequence with bad pages")
        want, _, tol, _ = R.attend(q[n:], cache.rows("k", 1), cache.rows("v", 1), 100 - n, 0.125, True, 0)
        R.assert_within(out[n:], want, tol, "its neighbour")
        x = torch.randn(2 * n, 2, 64).bfloat16().to(DEV)
        kept = pk.k.clone()
        b2 = pk.batch(R.starts([n, n]).to(DEV), torch.tensor([n, n], dtype=torch.int32, device=DEV), table.to(DEV), 2 * n, n)
        pk.append(x, x, b2, ws)
        assert B.lmoe_last_device_status(ws) == B.LMOE_ERR_DEVICE_CHECK
        pages = set(table[0, 2:].tolist()) | set(table[1].tolist())
        for pg in range(cache.n_pages):
            if pg not in pages:
                assert torch.equal(pk.k[pg].view(torch.uint8), kept[pg].view(torch.uint8))


@pytest.mark.parametrize("what", ["order", "rows", "new", "length", "negative"])
def test_a_bad_sequence_is_left_out(what):
    for n in (2, 60):
        cache = R.Cache("int8", 1, 64, 16, [64, 64])
        pk = paged(cache, 2, 1, 64)
        ws = pk.workspace()
        starts, lens, max_new = R.starts([n, n]), torch.tensor([64, 64], dtype=torch.int32), n
        if what == "order":
            starts[2] = n - 1
        elif what == "rows":
            starts[2] = 2 * n + 1
            max_new = n + 1
        elif what == "new":
            starts[1] = n - 1        # the second has one more than max_new
        elif what == "length":
            lens[1] = 1 << 30
        else:
            lens[1] = -1
        out = torch.full((2 * n, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
        q = torch.randn(2 * n, 2, 64).bfloat16()
        pk.attend(q.to(DEV), pk.batch(starts.to(DEV), lens.to(DEV), cache.table.to(DEV), 2 * n, max_new), ws, out=out)
        assert B.lmoe_last_device_status(ws) == B.LMOE_ERR_DEVICE_CHECK
        m = starts[1].item()
        want, _, tol, _ = R.attend(q[:m], cache.rows("k", 0), cache.rows("v", 0), 64 - m, 0.125, True, 0)
        R.assert_within(out[:m], want, tol, "the good sequence")
        assert (out[m:] == 5.0).all()


# ----------------------------------------------------------------------------
# the gated delta rule
# ----------------------------------------------------------------------------

def delta_inputs(T, H, Hq, DK, DV, seed, decay="usual", l2norm=False):
    g = torch.Generator().manual_seed(seed)
    q, k = torch.randn(T, Hq, DK, generator=g), torch.randn(T, Hq, DK, generator=g)
    if not l2norm:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    v = torch.randn(T, H, DV, generator=g)
    if decay == "usual":
        ld = -torch.exp(torch.randn(T, H, generator=g) - 3)
    elif decay == "none":
        ld = torch.zeros(T, H)
    else:                         # from nothing forgotten to everything
        ld = -torch.exp(4 * torch.randn(T, H, generator=g))
        ld[torch.rand(T, H, generator=g) < 0.05] = -math.inf
    return q.bfloat16(), k.bfloat16(), v.bfloat16(), ld, torch.rand(T, H, generator=g)


def check_delta(H, Hq, DK, DV, ns, l2norm, decay="usual", seed=0, pad=0, src=None, dst=None, n_states=None, max_new=None):
    B_, T = len(ns), sum(ns)
    n_states = 2 * B_ + 1 if n_states is None else n_states
    src = list(range(B_)) if src is None else src
    dst = list(range(B_, 2 * B_)) if dst is None else dst
    q, k, v, ld, beta = delta_inputs(T + pad, H, Hq, DK, DV, seed, decay, l2norm)
    S = torch.randn(n_states, H, DK, DV, generator=torch.Generator().manual_seed(seed + 1))
    st = mixers.DeltaStates(H, Hq, DK, DV, l2norm=l2norm, state=S.to(DEV))
    mx = max(ns) if max_new is None else max_new
    ws = st.workspace(T + pad, B_, mx)
    ints = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (src, dst)]
    b = st.batch(R.starts(ns).to(DEV), *ints, n_tokens=T + pad, max_new=mx)
    out = torch.full((T + pad, H, DV), 5.0, dtype=torch.bfloat16, device=DEV)
    st.forward(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), beta.to(DEV), b, ws, out=out)
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK
    t0, want_S = 0, S.double()
    for s, n in enumerate(ns):
        w = slice(t0, t0 + n)
        S0 = S[src[s]] if src[s] >= 0 else torch.zeros(H, DK, DV)
        o, S1 = R.delta(q[w], k[w], v[w], ld[w], beta[w], S0, DK ** -0.5, l2norm)
        # a state row is a sum of up to DK + n fp32 terms, each carried through at most n steps that contract
        # (0 <= beta <= 1, |k| <= 1, decay <= 1): errors add up like the square root of their number; 8 of those
        mag = S1.abs().amax((1, 2)).clamp_min(1.0)
        tol_S = 8 * R.U_F32 * math.sqrt(DK + n) * 4 * mag
        if n:
            err = 8 * R.U_F32 * math.sqrt(DK + n) * 4 * mag * math.sqrt(DK) * DK ** -0.5
            # the output's own products take operands of 16 bits at the least (2^-17, over DK + 64 terms)
            mid = 2.0 ** -16 * o.abs().amax((0, 2)).clamp_min(mag * DK ** -0.5)
            R.assert_within(out[w], o, R.U_BF16 * 1.01 * o.abs() + (err + mid)[None, :, None], f"out of sequence {s}")
        if dst[s] >= 0:
            R.assert_within(st.state[dst[s]], S1, tol_S[:, None, None], f"state of sequence {s}")
            want_S[dst[s]] = math.nan
        t0 += n
    assert (out[T:] == 5.0).all()
    kept = ~torch.isnan(want_S)
    assert torch.equal(st.state.double().cpu()[kept], want_S[kept])
    return st


@pytest.mark.parametrize("l2norm", [False, True])
@pytest.mark.parametrize("H,Hq,DK,DV", [(2, 1, 64, 64), (4, 2, 128, 128), (3, 3, 64, 128), (2, 2, 128, 64)])
@pytest.mark.parametrize("ns", [[1], [4, 1, 3], [8, 0, 5], [9]])
def test_delta_few_tokens(H, Hq, DK, DV, ns, l2norm):
    check_delta(H, Hq, DK, DV, ns, l2norm, seed=DK + DV, pad=1)


@pytest.mark.parametrize("decay", ["usual", "none", "wide"])
@pytest.mark.parametrize("H,Hq,DK,DV", [(2, 1, 64, 64), (4, 2, 128, 128), (3, 3, 64, 128), (2, 2, 128, 64)])
@pytest.mark.parametrize("ns", [[64], [65, 1, 200], [0, 300, 63], [17, 128]])
def test_delta_prompts(H, Hq, DK, DV, ns, decay):
    check_delta(H, Hq, DK, DV, ns, True, decay, seed=DK + DV, pad=2)


@pytest.mark.parametrize("n", [3, 100])
def test_delta_states_by_place(n):
    """From zeros, in place, and to nowhere."""
    check_delta(2, 1, 64, 64, [n, n, n], False, src=[-1, 1, 2], dst=[0, 1, -1], n_states=4)


@pytest.mark.parametrize("n", [2, 70])
def test_delta_bad_sequences_are_left_out(n):
    H, DK = 2, 64
    q, k, v, ld, beta = delta_inputs(3 * n, H, H, DK, DK, 3)
    S = torch.randn(3, H, DK, DK)
    for case in ("src", "dst", "rows"):
        st = mixers.DeltaStates(H, H, DK, DK, state=S.to(DEV))
        ws = st.workspace(3 * n, 3, n)
        src, dst, qs = [0, 1, 2], [0, 1, 2], R.starts([n, n, n])
        if case == "src":
            src[1] = 3
        elif case == "dst":
            dst[1] = -2
        else:
            qs[2] = 2 * n + 1          # the second has more than max_new, the third fewer
        out = torch.full((3 * n, H, DK), 5.0, dtype=torch.bfloat16, device=DEV)
        b = st.batch(qs.to(DEV), *[torch.tensor(x, dtype=torch.int32, device=DEV) for x in (src, dst)], n_tokens=3 * n, max_new=n)
        st.forward(*[x.to(DEV) for x in (q, k, v, ld, beta)], b, ws, out=out)
        assert B.lmoe_last_device_status(ws) == B.LMOE_ERR_DEVICE_CHECK
        end = qs[2].item()
        assert (out[n:end] == 5.0).all() and not (out[:n] == 5.0).all() and not (out[end:] == 5.0).all()
        assert torch.equal(st.state[1].cpu(), S[1])


# ----------------------------------------------------------------------------
# streams, graphs
# ----------------------------------------------------------------------------

def test_another_stream_and_a_replayed_graph_with_other_lengths():
    cache = R.Cache("int8", 2, 128, 16, [300, 200])
    pk = paged(cache, 4, 2, 128)
    ws = pk.workspace()
    q = torch.randn(2, 4, 128).bfloat16()
    dq, lens, table = q.to(DEV), torch.tensor([300, 200], dtype=torch.int32, device=DEV), cache.table.to(DEV)
    b = pk.batch(R.starts([1, 1]).to(DEV), lens, table, 2, 1)
    out = torch.empty(2, 4, 128, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pk.attend(dq, b, ws, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pk.attend(dq, b, ws, out=out)
    for pair in ([300, 200], [17, 1], [256, 128]):
        lens.copy_(torch.tensor(pair, dtype=torch.int32))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for s in range(2):
            want, _, tol, _ = R.attend(q[s:s + 1], cache.rows("k", s, pair[s]), cache.rows("v", s, pair[s]), pair[s] - 1, 128 ** -0.5, True, 0)
            R.assert_within(out[s:s + 1], want, tol, f"lengths {pair}")


def graphed(step):
    """step() captured on a side stream, after one eager run."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    return graph


@pytest.mark.parametrize("n", [70, 150])
def test_a_replayed_graph_of_prompt_chunks(n):
    """Attention of many rows (one row tile, and more than four) and the chunked delta rule, replayed with other lengths."""
    cache = R.Cache("e4m3", 1, 64, 16, [400, 300])
    pk = paged(cache, 8, 1, 64)
    ws = pk.workspace()
    q = torch.randn(2 * n, 8, 64, generator=torch.Generator().manual_seed(n)).bfloat16()
    dq, table = q.to(DEV), cache.table.to(DEV)
    starts, lens = R.starts([n, n]).to(DEV), torch.tensor([400, 300], dtype=torch.int32, device=DEV)
    b = pk.batch(starts, lens, table, 2 * n, n)
    out = torch.empty(2 * n, 8, 64, dtype=torch.bfloat16, device=DEV)
    H, DK = 2, 64
    x = delta_inputs(2 * n, H, 1, DK, DK, 5, l2norm=True)
    S = torch.randn(2, H, DK, DK, generator=torch.Generator().manual_seed(6))
    st = mixers.DeltaStates(H, 1, DK, DK, l2norm=True, state=torch.cat([S, S]).to(DEV))
    dws = st.workspace(2 * n, 2, n)
    dx = [t.to(DEV) for t in x]
    src, dst = (torch.tensor(i, dtype=torch.int32, device=DEV) for i in ([0, 1], [2, 3]))
    db = st.batch(starts, src, dst, 2 * n, n)
    dout = torch.empty(2 * n, H, DK, dtype=torch.bfloat16, device=DEV)

    def step():
        pk.attend(dq, b, ws, out=out)
        st.forward(*dx, db, dws, out=dout)

    graph = graphed(step)
    for ns, kv in (([n, n], [400, 300]), ([n, 1], [n, 17]), ([3, n - 5], [400, 299])):
        starts.copy_(R.starts(ns))
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        out.fill_(5.0)
        dout.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        t0 = 0
        for s, m in enumerate(ns):
            w = slice(t0, t0 + m)
            want, _, tol, _ = R.attend(q[w], cache.rows("k", s, kv[s]), cache.rows("v", s, kv[s]), kv[s] - m, 0.125, True, 0)
            R.assert_within(out[w], want, tol, f"attention of sequence {s}, {m} rows")
            o, S1 = R.delta(*(t[w] for t in x), S[s], DK ** -0.5, True)
            # outputs: as in check_delta; the state carries fp32's errors alone (three-term operands)
            mag = S1.abs().amax()
            R.assert_within(dout[w], o, R.U_BF16 * 1.01 * o.abs() + 2.0 ** -14 * mag, f"delta rule of sequence {s}")
            R.assert_within(st.state[2 + s], S1, 32 * R.U_F32 * math.sqrt(DK + m) * mag * torch.ones_like(S1), f"state {s}")
            t0 += m
        assert (out[t0:] == 5.0).all() and (dout[t0:] == 5.0).all()
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK and B.lmoe_last_device_status(dws) == B.LMOE_OK


def test_two_streams_with_a_workspace_each():
    cache = R.Cache("int8", 2, 128, 16, [500])
    pk = paged(cache, 20, 2, 128)
    q = torch.randn(120, 20, 128, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    b = batch_of(pk, cache, [120])
    want = pk.attend(q, b, pk.workspace())
    streams, wss = [torch.cuda.Stream() for _ in range(2)], [pk.workspace() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(pk.attend(q, b, wss[i]))
    torch.cuda.synchronize()
    for g in got[0] + got[1]:
        assert torch.equal(g.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_layers_steps(fmt):
    """As a model runs them: a prompt in two chunks, then a verify window and single tokens, each appended and then
    attended to; and the states of a delta layer carried through the same steps."""
    Hq, Hk, D, page = 8, 2, 128, 32
    g = torch.Generator().manual_seed(3)
    lens = [0, 0]
    total = 200
    cache = R.Cache(fmt, Hk, D, page, [total, total], seed=4)
    cache.table = cache.table.clone()
    pk = paged(cache, Hq, Hk, D)
    ws = pk.workspace()
    H, DK = 4, 64
    st = mixers.DeltaStates(H, 2, DK, DK, n_states=2, l2norm=True, device=DEV)
    S = torch.zeros(2, H, DK, DK, dtype=torch.float64)
    place = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    from_zero = torch.tensor([-1, -1], dtype=torch.int32, device=DEV)
    for step, ns in enumerate(([100, 40], [33, 64], [4, 4], [1, 1], [1, 0])):
        T = sum(ns)
        lens = [a + n for a, n in zip(lens, ns)]
        qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g).bfloat16()
        d = qkv.to(DEV)
        b = batch_of(pk, cache, ns, lens=lens)
        pk.append(d[:, Hq:Hq + Hk], d[:, Hq + Hk:], b, ws)
        out = pk.attend(d[:, :Hq], b, ws)
        back = pk.read(b, ws)
        dws = st.workspace(T, 2, max(ns))
        x = delta_inputs(T, H, 2, DK, DK, 10 + step, l2norm=True)
        dout = st.forward(*(t.to(DEV) for t in x), st.batch(R.starts(ns).to(DEV), place if step else from_zero, place, T, max(ns)), dws)
        t0 = 0
        for s, n in enumerate(ns):
            w = slice(t0, t0 + n)
            for name, i in (("k", Hq), ("v", Hq + Hk)):
                cache.put(name, s, range(lens[s] - n, lens[s]), qkv[w, i:i + Hk])
            K, V = cache.rows("k", s, lens[s]), cache.rows("v", s, lens[s])
            for y, want in zip(back, (K, V)):
                if n:
                    R.assert_within(y[w], want[lens[s] - n:], R.U_BF16 * want[lens[s] - n:].abs() * (1 + 2.0 ** -20), "read back")
            if n:
                want, _, tol, _ = R.attend(qkv[w, :Hq], K, V, lens[s] - n, D ** -0.5, True, 0)
                R.assert_within(out[w], want, tol, f"step {step}, attention of sequence {s}")
            o, S[s] = R.delta(*(t[w] for t in x), S[s], DK ** -0.5, True)
            mag = S[s].abs().amax()
            if n:
                R.assert_within(dout[w], o, R.U_BF16 * 1.01 * o.abs() + 2.0 ** -14 * mag, f"step {step}, delta rule of sequence {s}")
            # every step's errors are fp32 roundings of a sum that contracts
            R.assert_within(st.state[s], S[s], 64 * R.U_F32 * math.sqrt(DK + lens[s]) * mag * torch.ones_like(S[s]), f"step {step}, state {s}")
            t0 += n
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK


@pytest.mark.parametrize("ns", [[1, 16], [300, 17, 64]])
def test_delta_states_keep_fp32(ns):
    """Operands of 16 bits would leave 2^-18 in the state; fp32's own steps leave a tenth of that."""
    H, Hq, DK, DV = 4, 2, 128, 128
    T = sum(ns)
    x = delta_inputs(T, H, Hq, DK, DV, 21, l2norm=True)
    S = torch.randn(len(ns), H, DK, DV, generator=torch.Generator().manual_seed(22))
    st = mixers.DeltaStates(H, Hq, DK, DV, l2norm=True, state=S.to(DEV))
    ws = st.workspace(T, len(ns), max(ns))
    place = torch.arange(len(ns), dtype=torch.int32, device=DEV)
    st.forward(*(t.to(DEV) for t in x), st.batch(R.starts(ns).to(DEV), place, place, T, max(ns)), ws)
    t0 = 0
    for s, n in enumerate(ns):
        _, want = R.delta(*(t[t0:t0 + n] for t in x), S[s], DK ** -0.5, True)
        got = st.state[s].double().cpu()
        # relative error in the mean: sqrt(4 roundings of half a step a chunk, at most 10 chunks remembered) < 2^-20.7
        assert (got - want).norm() / want.norm() < 2.0 ** -20.7
        t0 += n


def test_a_loose_bound_of_new_tokens():
    """max_new far above what any sequence has (a program that does not count) costs no more than n_tokens does."""
    check_delta(2, 1, 64, 64, [40, 3], True, max_new=1 << 30)
    check_attend("int8", 4, 2, 64, 16, [40, 3], [90, 3], max_new=1 << 30)
