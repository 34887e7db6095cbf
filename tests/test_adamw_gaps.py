"""Lists with None in a tensor's place: the copies' list alone may hold them."""

import pytest
import torch

import block_scaled_precision_gemm_gb300 as bsmm


@pytest.fixture(scope="module")
def lists():
    import __graft_entry__
    __graft_entry__.build()
    return bsmm._lists()


def test_addresses_of_nothing(lists):
    where, sizes, kind = lists.addresses([None, None], -1, None, 1, True)
    assert where == sizes == bytes(16) and kind is None
    assert lists.addresses([None], -1, None, 1, False) is None


def test_refusals(lists):
    p, z = [torch.zeros(5), torch.zeros(7)], torch.zeros
    for name in ("grads", "m", "v"):
        kw = {"grads": p, "m": p, "v": p, name: [None, p[1]]}
        with pytest.raises((TypeError, ValueError), match="Tensors|CUDA"):
            bsmm.adamw(p, step=1, lr=0.1, **kw)
    with pytest.raises(TypeError, match="copies must hold"):
        bsmm._tensor_list([None, 1.0], "copies", None, dtypes=(torch.bfloat16,), gaps=True)
    with pytest.raises(ValueError, match="copies must be torch.bfloat16"):
        bsmm._tensor_list([None, z(7)], "copies", None, dtypes=(torch.bfloat16,), gaps=True)
    sizes = (5).to_bytes(8, "little") + (7).to_bytes(8, "little")
    with pytest.raises(ValueError, match=r"copies\[1\] holds 6 numbers, 7 needed"):
        bsmm._tensor_list([None, z(6).bfloat16()], "copies", sizes, dtypes=(torch.bfloat16,), gaps=True)
    with pytest.raises(ValueError, match="copies holds 1 tensors, 2 needed"):
        bsmm._tensor_list([None], "copies", sizes, dtypes=(torch.bfloat16,), gaps=True)
    with pytest.raises(ValueError, match="CUDA"):
        bsmm._tensor_list([None, z(7).bfloat16()], "copies", sizes, dtypes=(torch.bfloat16,), gaps=True)


@pytest.mark.gpu
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("which", [(), (0,), (1, 3), (0, 1, 2, 3)])
def test_copies_where_they_are_given(lists, bits8, which):
    """The same parameters with and without, and copies of those asked for."""
    sizes = [5000, 7, 300, 4096]

    def made():
        g = torch.Generator("cuda").manual_seed(1)
        d = {"params": [torch.randn(n, device="cuda", generator=g) for n in sizes],
             "grads": [torch.randn(n, device="cuda", generator=g) for n in sizes]}
        for k in ("m", "v"):
            d[k] = [torch.zeros(n, device="cuda", dtype=torch.uint8 if bits8 else torch.float32) for n in sizes]
            if bits8:
                d[k + "_scales"] = [torch.zeros((n + 127) // 128, device="cuda") for n in sizes]
        return d

    a, b = made(), made()
    bsmm.adamw(**a, step=1, lr=0.1)
    copies = [torch.zeros(n, device="cuda", dtype=torch.bfloat16) if i in which else None for i, n in enumerate(sizes)]
    before = [t._version for t in b["params"]]
    bsmm.adamw(**b, step=1, lr=0.1, copies=copies)
    for i in range(len(sizes)):
        assert torch.equal(a["params"][i], b["params"][i]) and b["params"][i]._version > before[i]
        if i in which:
            assert torch.equal(copies[i], b["params"][i].bfloat16())
