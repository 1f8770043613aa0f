"""Host side of the token mixers: shapes, sizes and refusals, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from latent_mixture_experts_softmax_b200 import binding as B
from latent_mixture_experts_softmax_b200 import build, mixers

import mixers_ref as R


@pytest.fixture(scope="module")
def L():
    build.build_all()
    return B.lib()


def test_shapes(L):
    ok = dict(n_heads=20, n_kv_heads=4, head_dim=128, page_size=64, kv_fmt=B.LMOE_KV_INT8)
    assert B.lmoe_attn_cfg_check(B.lmoe_attn_cfg(**ok)) == B.LMOE_OK
    assert B.lmoe_attn_workspace_bytes(B.lmoe_attn_cfg(**ok)) > 4096
    for bad in (dict(n_heads=21), dict(head_dim=96), dict(head_dim=512), dict(page_size=48), dict(page_size=8),
                dict(page_size=2048), dict(kv_fmt=2), dict(n_heads=2048)):
        cfg = B.lmoe_attn_cfg(**{**ok, **bad})
        assert B.lmoe_attn_cfg_check(cfg) == B.LMOE_ERR_UNSUPPORTED, bad
        assert B.lmoe_attn_workspace_bytes(cfg) == 0
    for bad in (dict(n_heads=0), dict(n_kv_heads=-1), dict(page_size=0)):
        assert B.lmoe_attn_cfg_check(B.lmoe_attn_cfg(**{**ok, **bad})) == B.LMOE_ERR_ARG, bad
    assert L.lmoe_attn_cfg_check(None) == B.LMOE_ERR_ARG
    ok = dict(n_heads=32, n_qk_heads=16, head_k=128, head_v=128, l2norm=1)
    assert B.lmoe_delta_cfg_check(B.lmoe_delta_cfg(**ok)) == B.LMOE_OK
    assert B.lmoe_delta_workspace_bytes(B.lmoe_delta_cfg(**ok), 4, 1, 4) >= 4096
    assert B.lmoe_delta_workspace_bytes(B.lmoe_delta_cfg(**ok), -1, 1, 4) == 0
    for bad in (dict(n_heads=33), dict(head_k=96), dict(head_v=256)):
        assert B.lmoe_delta_cfg_check(B.lmoe_delta_cfg(**{**ok, **bad})) == B.LMOE_ERR_UNSUPPORTED, bad
    assert L.lmoe_delta_cfg_check(None) == B.LMOE_ERR_ARG


def test_attention_refusals(L):
    """(addresses are never followed: every call is refused before a launch)"""
    cfg = B.lmoe_attn_cfg(4, 2, 64, 16, 0)
    big = 1 << 40
    cache = B.lmoe_kv_cache(256, 256, 256, 256, 8)
    batch = B.lmoe_kv_batch(256, 256, 256, 2, 4, 6, 3)

    def attend(cfg=cfg, cache=cache, batch=batch, q=256, stride=256, scale=1.0, causal=1, window=0, out=256, lse=None, ws=256, n=big):
        return L.lmoe_attend(cfg, cache, batch, q, stride, scale, causal, window, out, lse, ws, n, None)

    def append(k=256, v=256, ks=128, vs=128, **kw):
        a = dict(cfg=cfg, cache=cache, batch=batch, ws=256, n=big, f=L.lmoe_kv_append) | kw
        return a["f"](a["cfg"], a["cache"], a["batch"], k, v, ks, vs, a["ws"], a["n"], None)

    for kw in (dict(cfg=None), dict(cache=None), dict(batch=None), dict(ws=None), dict(ws=128),
               dict(cache=B.lmoe_kv_cache(None, 256, 256, 256, 8)), dict(cache=B.lmoe_kv_cache(256, 264, 256, 256, 8)),
               dict(cache=B.lmoe_kv_cache(256, 256, 256, 260, 8)), dict(cache=B.lmoe_kv_cache(256, 256, 256, 256, 0)),
               dict(batch=B.lmoe_kv_batch(None, 256, 256, 2, 4, 6, 3)), dict(batch=B.lmoe_kv_batch(256, 258, 256, 2, 4, 6, 3)),
               dict(batch=B.lmoe_kv_batch(256, 256, 256, -1, 4, 6, 3)), dict(batch=B.lmoe_kv_batch(256, 256, 256, 2, 0, 6, 3)),
               dict(batch=B.lmoe_kv_batch(256, 256, 256, 2, 4, -6, 3)), dict(batch=B.lmoe_kv_batch(256, 256, 256, 2, 4, 6, -3))):
        assert attend(**kw) == B.LMOE_ERR_ARG, kw
        assert append(**kw) == B.LMOE_ERR_ARG, kw
        assert append(f=L.lmoe_kv_read, **kw) == B.LMOE_ERR_ARG, kw
    for kw in (dict(q=None), dict(q=264), dict(stride=248), dict(stride=260), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(window=-1), dict(window=4, causal=0), dict(out=None), dict(out=8), dict(lse=2)):
        assert attend(**kw) == B.LMOE_ERR_ARG, kw
    for kw in (dict(k=None), dict(v=264), dict(ks=120), dict(vs=132)):
        assert append(**kw) == B.LMOE_ERR_ARG, kw
        assert append(f=L.lmoe_kv_read, **kw) == B.LMOE_ERR_ARG, kw
    assert attend(n=4096) == B.LMOE_ERR_WORKSPACE and append(n=4096) == B.LMOE_ERR_WORKSPACE
    assert attend(cfg=B.lmoe_attn_cfg(4, 2, 80, 16, 0)) == B.LMOE_ERR_UNSUPPORTED
    # nothing to do
    for b in ((0, 4, 6, 3), (2, 4, 0, 3), (2, 4, 6, 0)):
        empty = B.lmoe_kv_batch(None, None, None, *b)
        assert attend(batch=empty, ws=None, q=None) == B.LMOE_OK and append(batch=empty, ws=None, k=None) == B.LMOE_OK


def test_delta_refusals(L):
    cfg = B.lmoe_delta_cfg(4, 2, 64, 64, 0)
    batch = B.lmoe_delta_batch(256, 256, 256, 2, 4, 6, 3)

    def go(cfg=cfg, batch=batch, q=256, k=256, v=256, qs=128, ks=128, vs=256, ld=256, beta=256, scale=1.0, st=256, out=256, ws=256, n=1 << 40):
        return L.lmoe_delta_rule(cfg, batch, q, k, v, qs, ks, vs, ld, beta, scale, st, out, ws, n, None)

    for kw in (dict(cfg=None), dict(batch=None), dict(q=None), dict(k=264), dict(vs=248), dict(qs=132), dict(ks=120), dict(ld=None),
               dict(beta=258), dict(scale=float("nan")), dict(st=None), dict(st=264), dict(out=None), dict(ws=None), dict(ws=64),
               dict(batch=B.lmoe_delta_batch(None, 256, 256, 2, 4, 6, 3)), dict(batch=B.lmoe_delta_batch(256, 256, 258, 2, 4, 6, 3)),
               dict(batch=B.lmoe_delta_batch(256, 256, 256, -2, 4, 6, 3)), dict(batch=B.lmoe_delta_batch(256, 256, 256, 2, -4, 6, 3))):
        assert go(**kw) == B.LMOE_ERR_ARG, kw
    assert go(n=100) == B.LMOE_ERR_WORKSPACE
    assert go(cfg=B.lmoe_delta_cfg(4, 3, 64, 64, 0)) == B.LMOE_ERR_UNSUPPORTED
    assert go(batch=B.lmoe_delta_batch(None, None, None, 0, 4, 6, 3), ws=None) == B.LMOE_OK


def test_sizes_that_no_launch_can_count_are_refused(L):
    cfg = B.lmoe_attn_cfg(8, 2, 64, 16, 0)
    many = B.lmoe_kv_batch(256, 256, 256, 1, 4, 2 ** 30, 2 ** 30)
    cache = B.lmoe_kv_cache(256, 256, 256, 256, 4)
    assert L.lmoe_attend(cfg, cache, many, 256, 512, 1.0, 1, 0, 256, None, 256, 1 << 40, None) == B.LMOE_ERR_UNSUPPORTED
    cfg = B.lmoe_delta_cfg(4, 2, 64, 64, 0)
    many = B.lmoe_delta_batch(256, 256, 256, 2 ** 30, 4, 6, 3)
    assert L.lmoe_delta_rule(cfg, many, 256, 256, 256, 128, 128, 256, 256, 256, 1.0, 256, 256, 256, 1 << 40, None) == B.LMOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("top", [127, 448])
def test_codes_by_reciprocals_are_those_of_exact_quotients(top):
    """The rule of the cache's write kernel (the product with the rounded reciprocal, to 20 bits, then to the codes'
    grid) in fp32, over every pair of bf16 significands and every shift that leaves a code, against integers."""
    X = np.arange(256, dtype=np.int64)
    for A in range(128, 256):
        inv = np.float32(1) / np.float32(A)
        for sh in range(20):
            x = X[X <= A << sh]
            y = (x.astype(np.float32) * np.float32(2.0 ** -sh) * np.float32(top)) * inv
            y = ((y.view(np.uint32) + np.uint32(8)) & np.uint32(0xFFFFFFF0)).view(np.float32).astype(np.float64)
            num, den = x * top, np.int64(A) << sh               # the quotient
            # the codes' steps: 1, or 2^(e - 3) in the binade e from -6 on (the largest power of two at most num / den)
            e = np.zeros_like(x) + 3 if top == 127 else np.full_like(x, -6)
            if top == 448:
                for i in range(-5, 9):
                    e[num * 2 ** max(0, -i) >= den * 2 ** max(0, i)] = i
            up, down = 2 ** np.maximum(0, 3 - e), 2 ** np.maximum(0, e - 3)
            k, r = np.divmod(num * up, den * down)
            k += (2 * r > den * down) | ((2 * r == den * down) & (k % 2 == 1))
            step = 2.0 ** (e - 3)
            assert np.array_equal(np.rint(y / step), k.astype(np.float64)), (A, sh)


def test_the_structures_have_the_headers_layout():
    for c, fields in ((B.lmoe_kv_cache, 4 * 8 + 8), (B.lmoe_kv_batch, 3 * 8 + 16), (B.lmoe_delta_batch, 3 * 8 + 16),
                      (B.lmoe_attn_cfg, 20), (B.lmoe_delta_cfg, 20)):
        assert ctypes.sizeof(c) == fields


def test_the_references_agree_with_plain_sums():
    """The 64-bit attention against an explicit loop, the encoder against torch's own 8-bit float."""
    torch.manual_seed(0)
    q, K, V = torch.randn(3, 4, 8).bfloat16(), torch.randn(6, 2, 8).double(), torch.randn(6, 2, 8).double()
    out, lse, _, _ = R.attend(q, K, V, 2, 0.3, True, 2)
    for i in range(3):
        for h in range(4):
            keys = [j for j in range(6) if 2 + i - 2 < j <= 2 + i]
            e = [torch.exp(0.3 * (q[i, h].double() @ K[j, h // 2])) for j in keys]
            want = sum(w * V[j, h // 2] for w, j in zip(e, keys)) / sum(e)
            assert torch.allclose(out[i, h], want) and torch.allclose(lse[i, h], sum(e).log())
    x = torch.randn(50, 64).bfloat16()
    c, s = R.encode(x, "e4m3")
    y = (x.double() * 448 / x.double().abs().amax(-1, keepdim=True)).float().to(torch.float8_e4m3fn)
    assert torch.equal(c.float(), y.float())
    assert torch.equal(s, x.float().abs().amax(-1) / 448)


def test_the_tensor_classes_refuse_what_does_not_fit():
    with pytest.raises(B.LmoeError):
        mixers.PagedKV(5, 2, 128, 64, 4)
    with pytest.raises(ValueError):
        mixers.PagedKV(4, 2, 128, 64, 4, device="cpu")
    with pytest.raises(B.LmoeError):
        mixers.DeltaStates(4, 3, 128, 128, 4)
    cache = R.Cache("int8", 2, 64, 16, [20])
    kv = mixers.PagedKV(4, 2, 64, 16, buffers=cache.buffers("cpu"))
    with pytest.raises(ValueError):
        mixers.PagedKV(4, 2, 64, 32, buffers=cache.buffers("cpu"))
    with pytest.raises(ValueError):
        mixers.PagedKV(4, 2, 64, 16, kv_fmt="e4m3", buffers=cache.buffers("cpu"))
    good = R.starts([3]), torch.tensor([20], dtype=torch.int32), cache.table
    b = kv.batch(*good, n_tokens=3, max_new=3)
    with pytest.raises(ValueError):
        kv.batch(good[0].long(), *good[1:], n_tokens=3, max_new=3)
    with pytest.raises(ValueError):
        kv.batch(good[0][:1], *good[1:], n_tokens=3, max_new=3)
    with pytest.raises(ValueError):
        kv.batch(good[0], good[1], cache.table[:, :1].expand(1, 2), n_tokens=3, max_new=3)
    ws = torch.zeros(4096, dtype=torch.uint8)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for bad in (q.float(), q[:2], q.transpose(1, 2), torch.zeros(3, 8, 64, dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError):
            kv.attend(bad, b, ws)
    with pytest.raises(ValueError):
        kv.attend(q, b, ws, out=torch.zeros(3, 4, 64))
    with pytest.raises(ValueError):
        kv.attend(q, b, ws, lse=torch.zeros(3, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        kv.append(q, q, b, ws)


def test_workspace_sizes_are_those_the_header_states(L):
    for d, mib in ((64, 83), (128, 102), (256, 102)):
        cfg = B.lmoe_attn_cfg(4, 2, d, 16, 0)
        assert mib - 1 < B.lmoe_attn_workspace_bytes(cfg) / 2 ** 20 <= mib + 0.1


@pytest.mark.parametrize("scale", [2.4e38, -3.3e38])
def test_a_softmax_scale_beyond_fp32_in_base_two_is_refused(L, scale):
    """The kernels work in powers of two: scale * log2(e) has to be finite as well."""
    cfg = B.lmoe_attn_cfg(4, 2, 64, 16, 0)
    cache, batch = B.lmoe_kv_cache(256, 256, 256, 256, 8), B.lmoe_kv_batch(256, 256, 256, 2, 4, 6, 3)
    assert L.lmoe_attend(cfg, cache, batch, 256, 256, scale, 1, 0, 256, None, 256, 1 << 40, None) == B.LMOE_ERR_ARG
    assert L.lmoe_attend(cfg, cache, batch, 256, 256, 2.3e38, 1, 0, 256, None, 256, 0, None) == B.LMOE_ERR_WORKSPACE
