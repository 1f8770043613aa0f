"""The token mixers at the ends of what their calls accept, on the GPU, against the 64-bit forms of tests/mixers_ref.py."""
import importlib.util
import math

import pytest
import torch

from latent_mixture_experts_softmax_b200 import binding as B
from latent_mixture_experts_softmax_b200 import build, mixers

import mixers_ref as R
from test_gpu_mixers import DEV, batch_of, check_attend, check_delta, delta_inputs, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_all()
    assert torch.cuda.is_available()


def attended(cache, Hq, Hk, D, q, ns, scale=None, **kw):
    """One call over the cache against the 64-bit form, out and lse."""
    pk = paged(cache, Hq, Hk, D)
    ws = pk.workspace()
    scale = D ** -0.5 if scale is None else scale
    lse = torch.full((sum(ns), Hq), 5.0, device=DEV)
    out = pk.attend(q.to(DEV), batch_of(pk, cache, ns), ws, scale=scale, lse=lse, **kw)
    t0 = 0
    for s, n in enumerate(ns):
        want, wl, tol, ltol = R.attend(q[t0:t0 + n], cache.rows("k", s), cache.rows("v", s), cache.kv[s] - n, scale,
                                       kw.get("causal", True), kw.get("window", 0))
        R.assert_within(out[t0:t0 + n], want, tol, f"out of sequence {s}")
        R.assert_within(lse[t0:t0 + n], wl, ltol, f"lse of sequence {s}")
        t0 += n
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK
    return out


# ----------------------------------------------------------------------------
# windows
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 1 << 20])
@pytest.mark.parametrize("Hq,Hk,D,ns,kv", [(4, 2, 128, [6], [3]), (8, 1, 64, [60], [25]), (4, 2, 64, [200, 5], [120, 5]),
                                           (4, 1, 256, [90], [40])])
def test_a_window_wider_than_any_cache(window, Hq, Hk, D, ns, kv):
    """Fewer places than new tokens and a window that means "no limit": position - window must not wrap."""
    check_attend("int8", Hq, Hk, D, 16, ns, kv, window=window, seed=D)


# ----------------------------------------------------------------------------
# the size of value rows
# ----------------------------------------------------------------------------

# new tokens and query heads per key head: 5, 15 and 30 rows, 80 (converted on the way), 600 and 1200 (images)
ROWS = [(5, 1), (5, 3), (6, 5), (40, 2), (150, 4), (300, 4)]


@pytest.mark.parametrize("fmt,D", [("int8", 128), ("e4m3", 256), ("int8", 64)])
@pytest.mark.parametrize("n,group", ROWS)
@pytest.mark.parametrize("size", [1e-8, 1.0, 1e20])
@pytest.mark.parametrize("zero_scale", [1.0, 0.0])
def test_value_rows_of_zeros(fmt, D, n, group, size, zero_scale):
    """A row of zeros adds to the sum of exponentials and to nothing else, whatever its scale says (1 as the cache
    stores it, 0 as other encoders do) and however much larger its score or smaller the other rows' values are: whole
    tiles of them, single ones, one whole sequence."""
    m = n + 100
    g = torch.Generator().manual_seed(n)
    cache = R.Cache(fmt, 1, D, 16, [m, m], seed=3)
    v = (torch.randn(m, 1, D, generator=g) * size).bfloat16()
    k = torch.randn(m, 1, D, generator=g)
    zero = torch.rand(m, generator=g) < 0.1
    zero[:70] = True
    zero[m - n // 2] = True
    v[zero] = 0
    k[zero] *= 3
    for s in range(2):
        cache.put("k", s, range(m), k.bfloat16())
        cache.put("v", s, range(m), v if s == 0 else torch.zeros_like(v))
    if zero_scale != 1.0:
        for s in range(2):
            for pos in range(m):
                if zero[pos] or s == 1:
                    cache.scale["v"][cache.table[s, pos // 16].item(), :, pos % 16] = zero_scale
    q = torch.randn(2 * n, group, D, generator=g).bfloat16()
    out = attended(cache, group, 1, D, q, [n, n])
    assert (out[n:] == 0).all()


@pytest.mark.parametrize("n,group", ROWS)
@pytest.mark.parametrize("D", [64, 256])
def test_a_scale_of_zero_makes_its_codes_zeros(D, n, group):
    """value = code * scale, codes that are not zero under a scale of 0 included."""
    cache = R.Cache("int8", 1, D, 16, [n + 90])
    g = torch.Generator().manual_seed(1)
    for pos in torch.randperm(n + 90, generator=g)[:30].tolist():
        cache.scale["v"][cache.table[0, pos // 16].item(), :, pos % 16] = 0.0
    attended(cache, group, 1, D, torch.randn(n, group, D, generator=g).bfloat16(), [n])


@pytest.mark.parametrize("bad", [-1.0, -0.03, math.inf, math.nan])
@pytest.mark.parametrize("codes", ["any", "zeros"])
@pytest.mark.parametrize("D,n,group", [(64, 6, 1), (256, 6, 5), (128, 40, 2), (64, 150, 4)])
def test_a_value_scale_that_is_no_number_from_zero_on_reaches_only_the_queries_that_see_it(bad, codes, D, n, group):
    m = n + 90
    cache = R.Cache("int8", 1, D, 16, [m], seed=n)
    g = torch.Generator().manual_seed(n)
    q = torch.randn(n, group, D, generator=g).bfloat16()
    at = m - n // 2
    page = cache.table[0, at // 16].item()
    if codes == "zeros":
        cache.codes["v"][page, :, at % 16] = 0.0
    K, V = cache.rows("k", 0), cache.rows("v", 0)
    cache.scale["v"][page, :, at % 16] = bad
    pk = paged(cache, group, 1, D)
    ws = pk.workspace()
    out = pk.attend(q.to(DEV), batch_of(pk, cache, [n]), ws)
    first = at - (m - n)                                 # the first query that sees it
    want, _, tol, _ = R.attend(q[:first], K[:at], V[:at], m - n, D ** -0.5, True, 0)
    R.assert_within(out[:first], want, tol, "queries before")
    assert torch.isnan(out[first:]).all()


@pytest.mark.parametrize("D,n,group", [(64, 5, 1), (256, 5, 3), (256, 6, 5), (128, 40, 2), (64, 150, 4), (256, 150, 4)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_under_a_scale_of_one(fmt, D, n, group):
    """A cache whose scales are all 1, as formats without scales have it, a few of its rows zeros: in their first
    bytes, in half of their columns, in all of them."""
    cache = R.Cache(fmt, 1, D, 16, [n + 150], seed=n)
    g = torch.Generator().manual_seed(n)
    for name in "kv":
        cache.scale[name][:] = 1.0
    cache.scale["k"] *= 0.02
    for i, pos in enumerate(torch.randperm(n + 150, generator=g)[:60].tolist()):
        row = cache.codes["v"][cache.table[0, pos // 16].item(), 0, pos % 16]
        row[slice(*((0, 20), (0, D // 2), (D // 2, D), (0, D))[i % 4])] = 0
    attended(cache, group, 1, D, torch.randn(n, group, D, generator=g).bfloat16(), [n])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,group", [(1, 4), (20, 4), (150, 4)])
@pytest.mark.parametrize("log2", [-100, -60, 90])
def test_value_rows_of_any_size(fmt, n, group, log2):
    """Long contexts of equal scores whose value rows are all very small or large: the sum of exponentials over the
    scales has to stay inside fp32."""
    m, D = 16384, 64
    g = torch.Generator().manual_seed(n)
    cache = R.Cache(fmt, 1, D, 1024, [m])
    v = (2 * torch.rand(m, 1, D, generator=g) - 1) * 2.0 ** log2
    v[:, :, 0] = 2.0 ** log2                     # (every row's largest: none is stored as zeros)
    cache.put("v", 0, range(m), v.bfloat16())
    attended(cache, group, 1, D, torch.zeros(n, group, D).bfloat16(), [n], causal=False)


@pytest.mark.parametrize("n,group", [(1, 4), (20, 4), (70, 4)])
def test_rising_scores_over_small_value_rows(n, group):
    """Scores that rise just too little to move the reference, over rows of 2^-100, in pieces of several key tiles."""
    m, D, Hk = 8192, 64, 4
    g = torch.Generator().manual_seed(n)
    cache = R.Cache("e4m3", Hk, D, 1024, [m] * 4)
    v = (2 * torch.rand(m, Hk, D, generator=g) - 1) * 2.0 ** -100
    v[:, :, 0] = 2.0 ** -100
    k = torch.zeros(m, Hk, D)
    k[:, :, 0] = torch.where(torch.arange(m) % 512 < 128, 0.0, 6.0)[:, None]
    for s in range(4):
        cache.put("v", s, range(m), v.bfloat16())
        cache.put("k", s, range(m), k.bfloat16())
    q = torch.zeros(4 * n, Hk * group, D)
    q[:, :, 0] = 1
    attended(cache, Hk * group, Hk, D, q.bfloat16(), [n] * 4, scale=1.0, causal=False)


@pytest.mark.parametrize("n,group", ROWS)
def test_zeros_before_rows_of_other_sizes(n, group):
    """Rows of zeros come first, then rows of 2^-99, of 2^-20 and of 2^40 that only later queries see."""
    m, D = n + 200, 64
    g = torch.Generator().manual_seed(n)
    for sizes in ([0, 2.0 ** -98], [0, 2.0 ** -98, 2.0 ** -20], [0, 2.0 ** 40], [2.0 ** 40, 0]):
        cache = R.Cache("int8", 1, D, 16, [m])
        v = torch.randn(m, 1, D, generator=g)
        for i, x in enumerate(sizes):
            v[m * i // len(sizes):m * (i + 1) // len(sizes)] *= x
        cache.put("v", 0, range(m), v.bfloat16())
        attended(cache, group, 1, D, torch.randn(n, group, D, generator=g).bfloat16(), [n])


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("n,group", ROWS)
def test_queries_with_elements_of_unequal_size(D, n, group):
    """Elements far below their row's largest, where only these meet keys: off by 2^-25 of its power of two at most."""
    m = n + 60
    g = torch.Generator().manual_seed(n)
    cache = R.Cache("int8", 1, D, 16, [m])
    k = torch.randn(m, 1, D, generator=g) * 2.0 ** 14
    k[:, :, 0] = 0
    cache.put("k", 0, range(m), k.bfloat16())
    q = torch.randn(n, group, D, generator=g) * torch.exp2(-12 - 10 * torch.rand(n, group, D, generator=g))
    q[:, :, 0] = 1.5
    q = q.bfloat16()
    pk = paged(cache, group, 1, D)
    ws = pk.workspace()
    out = pk.attend(q.to(DEV), batch_of(pk, cache, [n]), ws)
    K, V = cache.rows("k", 0), cache.rows("v", 0)
    want, _, tol, _ = R.attend(q, K, V, m - n, D ** -0.5, True, 0)
    # every weight is off by twice the largest score's error, to first order, and a little for the second
    ds = D ** -0.5 * 2.0 ** -25 * K.abs().sum(-1).max()
    R.assert_within(out, want, tol + 2.2 * ds * V.abs().max(), "out")


# ----------------------------------------------------------------------------
# long contexts of single tokens
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,Hq,Hk,D,page,kv", [("int8", 5, 1, 128, 256, 9000), ("e4m3", 16, 1, 256, 1024, 6100),
                                                ("int8", 3, 1, 64, 1024, 20000), ("e4m3", 8, 2, 128, 256, 16000)])
def test_one_token_behind_a_long_context(fmt, Hq, Hk, D, page, kv):
    """An item in more than 32 parts."""
    check_attend(fmt, Hq, Hk, D, page, [1], [kv], seed=D)


# ----------------------------------------------------------------------------
# the gated delta rule and numbers that are not finite
# ----------------------------------------------------------------------------

def check_bad(n, H, Hq, DK, DV, spots, l2norm=True, seed=1):
    """Tokens before a bad number, and heads and columns that it does not reach, are what they are without it."""
    q, k, v, ld, beta = delta_inputs(n, H, Hq, DK, DV, seed, l2norm=l2norm)
    for what, at, value in spots:
        dict(q=q, k=k, v=v, decay=ld, beta=beta)[what][at] = value
    S = torch.randn(1, H, DK, DV, generator=torch.Generator().manual_seed(seed + 1))
    st = mixers.DeltaStates(H, Hq, DK, DV, l2norm=l2norm, state=S.to(DEV))
    place = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = st.forward(*(x.to(DEV) for x in (q, k, v, ld, beta)), st.batch(R.starts([n]).to(DEV), place, place, n, n), st.workspace(n, 1, n))
    o, S1 = R.delta(q, k, v, ld, beta, S[0], DK ** -0.5, l2norm)
    fine = torch.isfinite(o)
    assert torch.equal(torch.isfinite(out.cpu()), fine), "outputs that are finite"
    assert torch.equal(torch.isfinite(st.state[0].cpu()), torch.isfinite(S1)), "states that are finite"
    # bounds as for batches without bad numbers: a bf16 rounding, fp32's errors, operands of 16 bits
    mag = S[0].abs().amax().double().clamp_min(1.0) * 4
    tol = R.U_BF16 * 1.01 * o.abs() + 2.0 ** -14 * mag
    got = torch.where(fine, out.double().cpu(), 0.0)
    R.assert_within(got, torch.where(fine, o, 0.0), torch.where(fine, tol, 0.0), "out")
    some = torch.isfinite(S1)
    got = torch.where(some, st.state[0].double().cpu(), 0.0)
    R.assert_within(got, torch.where(some, S1, 0.0), torch.full_like(S1, 32 * R.U_F32 * math.sqrt(DK + n) * mag.item()), "state")


@pytest.mark.parametrize("H,Hq,DK,DV", [(2, 1, 64, 64), (4, 2, 128, 128), (3, 3, 64, 128), (2, 2, 128, 64)])
@pytest.mark.parametrize("n,at", [(4, 2), (16, 9), (16, 15), (1, 0), (100, 40), (100, 53), (64, 31), (70, 69)])
@pytest.mark.parametrize("what", ["q", "k", "v", "decay", "beta"])
def test_bad_numbers_reach_only_what_follows_them(H, Hq, DK, DV, n, at, what):
    place = {"q": (at, Hq - 1, 5), "k": (at, Hq - 1, 7), "v": (at, H - 1, 33), "decay": (at, H - 1), "beta": (at, H - 1)}[what]
    check_bad(n, H, Hq, DK, DV, [(what, place, math.nan)])


@pytest.mark.parametrize("n,at", [(4, 2), (16, 9), (100, 40), (100, 60)])
@pytest.mark.parametrize("what,value", [("v", math.inf), ("v", -math.inf), ("beta", math.inf), ("k", math.inf)])
def test_infinities_reach_only_what_follows_them(n, at, what, value):
    place = {"k": (at, 0, 7), "v": (at, 1, 33), "beta": (at, 1)}[what]
    check_bad(n, 2, 1, 64, 64, [(what, place, value)], l2norm=False)


@pytest.mark.parametrize("n", [16, 100])
def test_several_bad_numbers(n):
    check_bad(n, 4, 2, 128, 128, [("v", (n - 3, 0, 17), math.nan), ("v", (n // 2, 0, 18), math.inf), ("k", (n - 5, 1, 0), math.nan),
                                  ("beta", (n // 3, 1), math.nan), ("decay", (n // 4, 1), math.nan), ("q", (0, 0, 0), math.nan)])


@pytest.mark.parametrize("DK,DV", [(64, 64), (128, 128)])
@pytest.mark.parametrize("ns", [[17], [33, 63, 20], [95, 1, 31]])
def test_ragged_chunks_behind_bad_rows(DK, DV, ns):
    """What a chunk's missing rows hold is zeros, whatever stood in their place (rows of NaN, of the call before)."""
    n = 96
    st = mixers.DeltaStates(2, 1, DK, DV, n_states=8, l2norm=True, device=DEV)
    bad = [x.to(DEV) * math.nan for x in delta_inputs(8 * n, 2, 1, DK, DV, 1)]
    place = torch.arange(8, dtype=torch.int32, device=DEV)
    st.forward(*bad, st.batch(R.starts([n] * 8).to(DEV), place, place, 8 * n, n), st.workspace(8 * n, 8, n))
    check_delta(2, 1, DK, DV, ns, True, seed=DK, pad=3)


# ----------------------------------------------------------------------------
# streams
# ----------------------------------------------------------------------------

def test_results_of_a_call_on_another_stream_are_that_streams_memory():
    """A result allocated for the current stream may take memory that its earlier work still writes to."""
    n = 1201
    cache = R.Cache("int8", 8, 256, 1024, [n])
    pk = paged(cache, 8, 8, 256)
    ws = pk.workspace()
    b = batch_of(pk, cache, [n])
    st = mixers.DeltaStates(16, 16, 128, 128, n_states=1, device=DEV)
    db = st.batch(R.starts([n]).to(DEV), *(torch.zeros(1, dtype=torch.int32, device=DEV) for _ in "sd"), n, n)
    dws = st.workspace(n, 1, n)
    q = torch.randn(n, 8, 256, device=DEV).bfloat16()
    x = [t.to(DEV) for t in delta_inputs(n, 16, 16, 128, 128, 1)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        for call in (lambda: [pk.attend(q, b, ws, stream=stream)], lambda: pk.read(b, ws, stream=stream),
                     lambda: [st.forward(*x, db, dws, stream=stream)]):
            torch.cuda.empty_cache()
            results = call()
            side.synchronize()
            at, shape = {y.data_ptr() for y in results}, results[0].shape
            del results
            with torch.cuda.stream(side):     # the stream's next memory of this size is what they had
                assert torch.empty(shape, dtype=torch.bfloat16, device=DEV).data_ptr() in at


@pytest.mark.parametrize("stream", [0, "default"])
def test_the_default_stream_by_handle_and_by_object(stream):
    cache = R.Cache("int8", 2, 64, 16, [50])
    pk = paged(cache, 4, 2, 64)
    ws = pk.workspace()
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    out = pk.attend(q.to(DEV), batch_of(pk, cache, [3]), ws, stream=torch.cuda.default_stream() if stream else 0)
    want, _, tol, _ = R.attend(q, cache.rows("k", 0), cache.rows("v", 0), 47, 0.125, True, 0)
    R.assert_within(out, want, tol, "out")


def test_a_torch_without_the_short_ways_to_stream_and_device(monkeypatch):
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.find_spec(mixers.__name__)
    plain = importlib.util.module_from_spec(spec)        # (a copy of its own; the loaded module stays as it is)
    spec.loader.exec_module(plain)
    monkeypatch.undo()
    cache = R.Cache("int8", 2, 64, 16, [50])
    pk = plain.PagedKV(4, 2, 64, 16, buffers=cache.buffers(DEV))
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    side = torch.cuda.Stream()
    want, _, tol, _ = R.attend(q, cache.rows("k", 0), cache.rows("v", 0), 47, 0.125, True, 0)
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            out = pk.attend(q.to(DEV), batch_of(pk, cache, [3]), pk.workspace())
        stream.synchronize()
        R.assert_within(out, want, tol, "out")


@pytest.mark.parametrize("n,group", [(1, 5), (6, 5), (40, 2), (150, 4)])
def test_rows_behind_the_last_token_may_be_written_meanwhile(n, group):
    """Attention of one step while another stream appends the next step's rows to the same pages."""
    D, m, more = 256, 1000, 100
    cache = R.Cache("int8", 1, D, 64, [m + more])
    pk = paged(cache, group, 1, D)
    wss = [pk.workspace() for _ in range(2)]
    g = torch.Generator().manual_seed(n)
    q = torch.randn(n, group, D, generator=g).bfloat16()
    dq = q.to(DEV)
    rows = [(torch.randn(more, 1, D, generator=g) * (i % 3)).bfloat16().to(DEV) for i in range(6)]     # rows of zeros as well
    now, after = batch_of(pk, cache, [n], lens=[m]), batch_of(pk, cache, [more])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(30):
        with torch.cuda.stream(streams[0]):
            got.append(pk.attend(dq, now, wss[0]))
        with torch.cuda.stream(streams[1]):
            for _ in range(4):
                pk.append(rows[i % 6], rows[(i + 1) % 6], after, wss[1])
    torch.cuda.synchronize()
    want, _, tol, _ = R.attend(q, cache.rows("k", 0, m), cache.rows("v", 0, m), m - n, D ** -0.5, True, 0)
    for out in got:
        R.assert_within(out, want, tol, "out")
    assert B.lmoe_last_device_status(wss[0]) == B.LMOE_OK and B.lmoe_last_device_status(wss[1]) == B.LMOE_OK


# ----------------------------------------------------------------------------
# offsets beyond 32 bits
# ----------------------------------------------------------------------------

def test_a_cache_of_more_than_four_gigabytes():
    Hk, D, page, pages = 2, 128, 64, 270000            # codes of 4.4 GB, keys and values each
    small = R.Cache("int8", Hk, D, page, [700, 300])
    at = torch.tensor([pages - 1 - i if i % 2 else i for i in range(small.n_pages)])
    table = torch.where(small.table >= 0, at[small.table.clamp_min(0).long()].int(), small.table)
    pk = mixers.PagedKV(8, Hk, D, page, n_pages=pages, device=DEV)
    ws = pk.workspace()
    for big, x in zip((pk.k, pk.v, pk.k_scale, pk.v_scale), small.buffers(DEV)):
        big[at.to(DEV)] = x
    g = torch.Generator().manual_seed(1)
    for ns in ([1, 1], [4, 2], [40, 3], [200, 300]):   # (8, 16, 160 and 1200 rows: each kernel)
        T = sum(ns)
        b = pk.batch(R.starts(ns).to(DEV), torch.tensor(small.kv, dtype=torch.int32, device=DEV), table.to(DEV), T, max(ns))
        x = torch.randn(T, 8 + 2 * Hk, D, generator=g).bfloat16()
        dx = x.to(DEV)
        pk.append(dx[:, 8:8 + Hk], dx[:, 8 + Hk:], b, ws)
        out, back = pk.attend(dx[:, :8], b, ws), pk.read(b, ws)
        t0 = 0
        for s, n in enumerate(ns):
            w = slice(t0, t0 + n)
            for name, i in (("k", 8), ("v", 8 + Hk)):
                small.put(name, s, range(small.kv[s] - n, small.kv[s]), x[w, i:i + Hk])
            K, V = small.rows("k", s), small.rows("v", s)
            for y, want in zip(back, (K, V)):
                R.assert_within(y[w], want[small.kv[s] - n:], R.U_BF16 * want[small.kv[s] - n:].abs() * (1 + 2.0 ** -20), "read back")
            want, _, tol, _ = R.attend(x[w, :8], K, V, small.kv[s] - n, D ** -0.5, True, 0)
            R.assert_within(out[w], want, tol, f"out of sequence {s}")
            t0 += n
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK


def test_states_of_more_than_four_gigabytes():
    H, DK, DV, places = 32, 128, 128, 2200             # 2 MB a state
    states = torch.zeros(places, H, DK, DV, device=DEV)
    st = mixers.DeltaStates(H, 16, DK, DV, l2norm=True, state=states)
    for ns in ([2, 1], [40, 17]):
        T = sum(ns)
        x = delta_inputs(T, H, 16, DK, DV, T, l2norm=True)
        src, dst = [places - 1, 3], [5, places - 2]
        S = torch.randn(2, H, DK, DV, generator=torch.Generator().manual_seed(T))
        states[src] = S.to(DEV)
        ints = [torch.tensor(i, dtype=torch.int32, device=DEV) for i in (src, dst)]
        out = st.forward(*(y.to(DEV) for y in x), st.batch(R.starts(ns).to(DEV), *ints, T, max(ns)), st.workspace(T, 2, max(ns)))
        t0 = 0
        for s, n in enumerate(ns):
            w = slice(t0, t0 + n)
            o, S1 = R.delta(*(y[w] for y in x), S[s], DK ** -0.5, True)
            mag = S1.abs().amax()
            R.assert_within(out[w], o, R.U_BF16 * 1.01 * o.abs() + 2.0 ** -14 * mag, f"out of sequence {s}")
            R.assert_within(states[dst[s]], S1, 32 * R.U_F32 * math.sqrt(DK + n) * mag * torch.ones_like(S1), f"state {s}")
            t0 += n


# ----------------------------------------------------------------------------
# two rows at one place
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_two_rows_at_one_place_touch_nothing_else(fmt):
    """Two sequences that share a page they write to: the place gets codes and scales of these rows (it is not said
    which), every other place is as without."""
    Hk, D, n = 2, 64, 9
    cache = R.Cache(fmt, Hk, D, 16, [40, 40])
    shared = cache.table.clone()
    shared[1, 2] = shared[0, 2]
    pk = paged(cache, Hk, Hk, D)
    ws = pk.workspace()
    x = torch.randn(2 * n, Hk, D, generator=torch.Generator().manual_seed(2)).bfloat16()
    b = pk.batch(R.starts([n, n]).to(DEV), torch.tensor([40, 40], dtype=torch.int32, device=DEV), shared.to(DEV), 2 * n, n)
    pk.append(x.to(DEV), x.to(DEV), b, ws)
    assert B.lmoe_last_device_status(ws) == B.LMOE_OK
    codes, scale = R.encode(x, fmt)
    got_c, got_s = pk.k.float().cpu(), pk.k_scale.cpu()
    place = shared[0, 2].item()
    for i in range(1, n):             # positions 32 .. 39 of both
        c, s = got_c[place, :, i - 1], got_s[place, :, i - 1]
        assert ((c == codes[i]) | (c == codes[n + i])).all() and ((s == scale[i]) | (s == scale[n + i])).all()
    for s in range(2):
        cache.put("k", s, [31], x[[s * n]])
    for page in range(cache.n_pages):
        if page != place:
            assert torch.equal(pk.k[page].cpu().view(torch.uint8), cache.buffers("cpu")[0][page].view(torch.uint8))
            assert torch.equal(got_s[page].nan_to_num(-1), cache.scale["k"][page].nan_to_num(-1))
    assert torch.equal(pk.k[place, :, n - 1:].cpu().view(torch.uint8), cache.buffers("cpu")[0][place, :, n - 1:].view(torch.uint8))
