"""Capped scores at and beyond their cap: rows whose raw products are all -inf, and gradients
where 1 - tanh^2 is small, against the 64-bit reference and bounds of tests/attention_mod_bounds.py."""
import pytest
import torch

import numerically_stable_online_gb300 as smx
from tests import attention_mod_bounds as bounds
from tests import attention_mod_ref as ref
from tests.test_attention_mod import DEV, DT, make, slopes_of

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


def compare(q, k, v, d_o=None, **mods):
    scale = q.shape[-1] ** -0.5
    o, lse = smx.attention_mod_forward(q, k, v, **mods)
    seen, pos = ref.visible(q.shape[0], q.shape[2], k.shape[2], q.device,
                            **{x: mods[x] for x in ("causal", "q_doc", "k_doc", "k_len") if x in mods})
    want = bounds.reference(q, k, v, scale, seen, pos, mods.get("softcap", 0.0), mods.get("slopes"), d_o)
    got = {"o": o, "lse": lse}
    if d_o is not None:
        got.update(zip(("dq", "dk", "dv"), smx.attention_mod_backward(q, k, v, o, lse, d_o, **mods)))
    over = {x: ref.excess(got[x], *want[x]) for x in got}
    print({x: round(y, 3) for x, y in over.items()})
    assert all(y <= 1.0 for y in over.values()), over
    return got


@pytest.mark.parametrize("kernel,splits", [(0, 0), (1, 1), (1, 3), (2, 1), (2, 3)])
@pytest.mark.parametrize("n,D", [(6, 128), (40, 64), (300, 128)])
@pytest.mark.parametrize("cap", [5.0, 120.0])
@pytest.mark.parametrize("biased", [False, True])
def test_products_of_minus_infinity(built, kernel, splits, n, D, cap, biased):
    """A capped score of -inf is -cap, a number: rows that see nothing else (k_len 64), rows whose first blocks hold
    nothing else, and rows where such keys lie among others.  Finite bf16 inputs, their products past 32 bits."""
    B, H, U, m = 3, 2, 1, 400
    q, k, v, d_o, g = make(n + D, B, H, U, n, m, D, "bf16")
    q[:, :, :, 0] = 0.0
    q[:, :, : n // 2, 0] = -(2.0 ** 100)
    k[:, :, :, 0] = 0.0
    k[0, :, :64, 0] = 2.0 ** 100
    k[1, :, :230, 0] = 2.0 ** 100
    k[2, :, ::3, 0] = 2.0 ** 100
    mods = {"softcap": cap, "k_len": torch.tensor([64, m, m - 5], dtype=torch.int32, device=DEV)}
    if biased:
        mods["slopes"] = slopes_of(H)
    built.smx_debug_set_attention_mod(kernel, splits)
    compare(q, k, v, d_o, **mods)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,D", [(3, 64), (130, 64), (70, 128)])
def test_an_infinite_key_under_a_cap(dt, n, D):
    """An infinite element of k: the score is -cap, by every kernel, whole or in parts."""
    q, k, v, _, _ = make(n * D, 2, 2, 2, n, 250, D, dt)
    q[:, :, :, 0] = -q[:, :, :, 0].abs() - 1.0
    k[0, :, :130, 0] = float("inf")
    k[1, :, 100:, 0] = float("inf")
    compare(q, k, v, softcap=7.0)


@pytest.mark.parametrize("std,cap", [(20.0, 20.0), (60.0, 20.0), (150.0, 50.0), (30.0, 5.0), (3.0, 50.0)])
@pytest.mark.parametrize("n,m,D", [(150, 210, 64), (16, 16, 128), (300, 300, 128), (4, 3, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gradients_where_a_cap_saturates(std, cap, n, m, D, dt):
    """Raw scores up to several times the cap, rows of few keys and of many."""
    q, k, v, d_o, _ = make(int(std) + n, 2, 4, 2, n, m, D, dt, std=std)
    compare(q, k, v, d_o, causal=m >= n, softcap=cap)
    compare(q, k, v, d_o, causal=m >= n, softcap=cap, slopes=slopes_of(4))


@pytest.mark.parametrize("std,cap", [(3.0, 20.0), (3.0, 0.0), (20.0, 20.0)])
def test_dq_takes_two_roundings(std, cap):
    """In fp16 dS is rounded once and dq once, whether scores are capped or not.  A rounding to fp16 is off by a uniform
    part of half a step, 2^-11 / m of a value of mantissa m: over mantissas in [1, 2) with density 1 / (m ln 2) its root
    mean square is 2^-11 / sqrt(3) sqrt(3 / (8 ln 2)) = 2.07e-4, and errors of many independent terms add up as the
    terms do.  Two of them make 2.93e-4 of dq's norm, three 3.59e-4; the limit lies between."""
    q, k, v, d_o, _ = make(int(std + cap), 2, 4, 2, 512, 512, 64, "f16", std=std)
    o, lse = smx.attention_mod_forward(q, k, v, softcap=cap)
    dq = smx.attention_mod_backward(q, k, v, o, lse, d_o, softcap=cap)[0].double()
    seen, pos = ref.visible(2, 512, 512, q.device)
    want = bounds.reference(q, k, v, 0.125, seen, pos, cap, None, d_o)["dq"][0]
    off = float((dq - want).norm() / want.norm())
    print(off)
    assert off <= 3.25e-4
