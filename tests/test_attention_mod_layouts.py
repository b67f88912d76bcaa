"""Layouts that the attention with modified scores takes: q, k, v, o and the gradients as slices of one buffer in
any order of its dimensions.  Without a GPU: such a call passes every check (it ends at the missing device, as a
dense one does).  With one: real tensors of each layout give what dense ones give, and leave the rest alone."""
import pytest
import torch

import numerically_stable_online_gb300 as smx
from tests import attention_mod_ref as ref
from tests.test_attention_mod_args import (ALIAS, INVALID, UNSUPPORTED, at, backward, desc, forward, interleaved,
                                           prefix_desc, shared)

D = 64
ORDERS = ["brsh", "brhs", "bshr", "bhsr", "bhrs", "sbhr", "bsrh", "rbhs"]
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls with made-up addresses: no GPU wanted")


@pytest.fixture(scope="module")
def lib():
    from numerically_stable_online_gb300 import build

    build.build()
    return smx.library()


@no_gpu
def test_a_dense_call_passes_every_check(lib):
    """What is left is the device: the status that the layouts below are held to."""
    assert forward(lib, desc()) == UNSUPPORTED and backward(lib, desc()) == UNSUPPORTED
    assert shared(lib, prefix_desc()) == UNSUPPORTED
    assert UNSUPPORTED not in (INVALID, ALIAS)


@no_gpu
def test_packed_rows_pass_every_check(lib):
    """q, k, v (and dq, dk, dv) of grouped heads as pieces of the rows of one buffer."""
    hq, hkv, n = 4, 2, 16
    row = (hq + 2 * hkv) * D
    s = (n * row, D, row)
    p = desc(seq_q=n, **{x + "_stride": s for x in ("q", "k", "v", "dq", "dk", "dv")})
    ins = {"q": at(1), "k": at(1) + hq * D * 2, "v": at(1) + (hq + hkv) * D * 2}
    outs = {"dq": at(7), "dk": at(7) + hq * D * 2, "dv": at(7) + (hq + hkv) * D * 2}
    assert forward(lib, p, **ins) == UNSUPPORTED
    assert backward(lib, p, **ins, **outs) == UNSUPPORTED
    assert backward(lib, p, **ins, **dict(outs, dk=outs["dk"] - 2 * D)) == ALIAS


@no_gpu
@pytest.mark.parametrize("order", ORDERS)
def test_slices_of_one_buffer_pass_every_check(lib, order):
    b, rows, heads, slots = 2, 16, 4, 4
    stride, slot = interleaved(order, b, rows, heads, slots)
    names = ("q", "k", "v", "o", "do", "dq", "dk", "dv")
    p = desc(batch=b, heads_q=heads, heads_kv=heads, seq_q=rows, seq_k=rows, **{x + "_stride": stride for x in names})
    s = [at(1) + 2 * slot * i for i in range(slots)]
    g = [at(3) + 2 * slot * i for i in range(slots)]
    assert forward(lib, p, q=s[0], k=s[1], v=s[2], o=s[3]) == UNSUPPORTED
    assert backward(lib, p, q=s[0], k=s[1], v=s[2], o=s[3], d_o=g[3], dq=g[0], dk=g[1], dv=g[2]) == UNSUPPORTED


def slots_of(order, b, rows, heads, slots, fill, dev):
    """(buffer, its slots as [batch, heads, rows, D] views) in the memory order `order`."""
    sizes = {"b": b, "r": rows, "h": heads, "s": slots}
    buffer = torch.full([sizes[x] for x in order] + [D], fill, dtype=torch.bfloat16, device=dev)
    view = buffer.permute(*(order.index(x) for x in "sbhr"), 4)
    return buffer, list(view)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("rows", [5, 150])
def test_slices_of_one_buffer_on_the_device(lib, order, rows):
    b, heads, dev = 2, 4, "cuda:0"
    g = torch.Generator(device=dev).manual_seed(rows)
    dense = [torch.randn(b, heads, rows, D, generator=g, device=dev).bfloat16() for _ in range(4)]
    buffer, s = slots_of(order, b, rows, heads, 4, 7.0, dev)
    for x, y in zip(s, dense[:3]):
        x.copy_(y)
    o, lse = smx.attention_mod_forward(s[0], s[1], s[2], causal=True, out=s[3])
    want, want_lse = smx.attention_mod_forward(*dense[:3], causal=True)
    assert o is s[3] and torch.equal(o, want) and torch.equal(lse, want_lse)
    assert all(torch.equal(x, y) for x, y in zip(s, dense[:3]))
    seen, pos = ref.visible(b, rows, rows, dev, causal=True)
    value = ref.reference(*dense[:3], D ** -0.5, seen, pos)
    assert ref.excess(o, *value["o"]) <= 1.0 and ref.excess(lse, *value["lse"]) <= 1.0
    grads, t = slots_of(order, b, rows, heads, 4, 7.0, dev)
    t[3].copy_(dense[3])
    smx.attention_mod_backward(s[0], s[1], s[2], o, lse, t[3], causal=True, dq=t[0], dk=t[1], dv=t[2])
    for x, y in zip(t, smx.attention_mod_backward(*dense[:3], want, want_lse, dense[3], causal=True)):
        assert torch.equal(x, y)
    assert torch.equal(t[3], dense[3])
