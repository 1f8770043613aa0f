"""The token mixers at the ends of what their calls accept, on the GPU, against the 64-bit forms of tests/mixers_ref.py."""
import math

import pytest
import torch

from latent_mixture_experts_softmax_b200 import binding as B
from latent_mixture_experts_softmax_b200 import build, mixers

import mixers_ref as R
from test_gpu_mixers import DEV, batch_of, check_attend, delta_inputs, paged

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
