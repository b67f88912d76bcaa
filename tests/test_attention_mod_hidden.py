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


def hidden_key(n, m, at):
    """Documents that hide key `at` from every query."""
    k_doc = torch.zeros(1, m, dtype=torch.int32, device=DEV)
    k_doc[:, at] = -1
    return {"q_doc": torch.zeros(1, n, dtype=torch.int32, device=DEV), "k_doc": k_doc}


def test_a_long_way_to_compute_again(built):
    """One hidden NaN among 16384 keys sends every row of the call the long way: 0.58 us a key, 0.3 s for a warp's 32
    rows, with a second item behind the first on some SMs.  No wait between a CTA's warps may run that long (they
    give up after 0.2 s), so the rows are computed again behind the last item."""
    H, n, m, D = 16, 2560, 16384, 64  # 160 items of 256 rows
    g = torch.Generator(device=DEV).manual_seed(8)
    q, k, v = normal(g, 1, H, n, D), normal(g, 1, H, m, D), normal(g, 1, H, m, D)
    v[:, :, m // 2] = float("nan")
    mods = hidden_key(n, m, m // 2)
    o, lse = smx.attention_mod_forward(q, k, v, **mods)
    torch.cuda.synchronize()
    assert smx.last_device_status() == 0
    rows = torch.tensor([0, 31, 32, 127, 128, 255, 1000, 2303, 2304, 2559], device=DEV)
    mods["q_doc"] = mods["q_doc"][:, rows]
    seen, pos = ref.visible(1, len(rows), m, q.device, **mods)
    want = bounds.reference(q[:, :, rows], k, v, D ** -0.5, seen, pos)
    over = {x: ref.excess(y[:, :, rows], *want[x]) for x, y in (("o", o), ("lse", lse))}
    assert all(y <= 1.0 for y in over.values()), over


@pytest.mark.parametrize("parts", [0, 1, 3])
@pytest.mark.parametrize("n,m,D,dt", [(300, 300, 64, "bf16"), (70, 1000, 128, "f16")])
def test_rows_of_many_items_computed_again(built, parts, n, m, D, dt):
    """More items than SMs, whole and in parts, each with rows to compute again; grouped heads."""
    B, H, U = 1, 320, 160
    g = torch.Generator(device=DEV).manual_seed(n)
    q, k, v = (normal(g, B, h, r, D, dt=DT[dt]) for h, r in ((H, n), (U, m), (U, m)))
    v[:, ::3, m // 3] = float("nan")
    k[:, 1::3, m // 3] = float("inf")
    mods = hidden_key(n, m, m // 3)
    built.smx_debug_set_attention_mod(0, parts)
    o, lse = smx.attention_mod_forward(q, k, v, causal=True, **mods)
    seen, pos = ref.visible(B, n, m, q.device, causal=True, **mods)
    want = bounds.reference(q, k, v, D ** -0.5, seen, pos)
    over = {x: ref.excess(y, *want[x]) for x, y in (("o", o), ("lse", lse))}
    assert all(y <= 1.0 for y in over.values()), over
