"""NaN in places that no row sees, where rows are computed again from the pairs they see: their gradients are
held to the same bounds as those of other rows (tests/attention_mod_bounds.py)."""
import pytest
import torch

import numerically_stable_online_gb300 as smx
from tests import attention_mod_bounds as bounds
from tests import attention_mod_ref as ref
from tests.test_attention_mod import DEV, DT, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from numerically_stable_online_gb300 import build

    build.build()
    yield smx.library()


@pytest.fixture(autouse=True)
def clean(built):
    yield
    built.smx_debug_set_attention_mod(0, 0)
    assert smx.last_device_status() == 0


@pytest.mark.parametrize("parts", [0, 2])
@pytest.mark.parametrize("where", ["nowhere", "v", "q", "all"])
@pytest.mark.parametrize("n,D,dt,cap", [(200, 64, "f16", 0.0), (140, 128, "bf16", 0.0), (140, 64, "f16", 9.0)])
def test_gradients_of_rows_beside_a_hidden_nan(built, parts, where, n, D, dt, cap):
    """Documents of 2 to 7 tokens whose values hardly differ, so that dP - D is far smaller than |do| |o| and an
    uncorrected D shows; places without a document hold NaN."""
    B, H = 2, 4
    g = torch.Generator(device=DEV).manual_seed(n + D)
    dtype = DT[dt]
    lengths = [2, 3, 7, 2, 5]
    doc = torch.cat([torch.full((x,), i, device=DEV) for i, x in enumerate(lengths * (n // 19 + 1))])[:n].int()
    doc[::23] = -1
    doc = doc.expand(B, n).contiguous()
    q, k, d_o = (normal(g, B, H, n, D, dt=dtype) for _ in range(3))
    v = (1.0 + torch.rand(B, H, 1, D, generator=g, device=DEV)).expand(B, H, n, D)
    v = (v + 2.0 ** -6 * torch.randn(B, H, n, D, generator=g, device=DEV)).to(dtype)
    hidden = (doc < 0)[:, None, :, None]
    if where in ("v", "all"):
        v = v.masked_fill(hidden, float("nan"))
    if where in ("q", "all"):
        q = q.masked_fill(hidden, float("nan"))
    if where == "all":
        k, d_o = k.masked_fill(hidden, float("nan")), d_o.masked_fill(hidden, float("nan"))
    mods = {"causal": True, "q_doc": doc, "k_doc": doc, "softcap": cap}
    built.smx_debug_set_attention_mod(0, parts)
    o, lse = smx.attention_mod_forward(q, k, v, **mods)
    got = dict(zip(("dq", "dk", "dv"), smx.attention_mod_backward(q, k, v, o, lse, d_o, **mods)), o=o, lse=lse)
    seen, pos = ref.visible(B, n, n, q.device, causal=True, q_doc=doc, k_doc=doc)
    want = bounds.reference(q, k, v, D ** -0.5, seen, pos, cap, None, d_o)
    over = {x: ref.excess(got[x], *want[x]) for x in got}
    print({x: round(y, 3) for x, y in over.items()})
    assert all(y <= 1.0 for y in over.values()), over
