"""Rows [T, heads, d] with one token or one head: the stride that is never used may be anything."""
import pytest
import torch

from chunk_wise_sparse_b200 import hils

pytestmark = pytest.mark.gpu

C = 64


def _odd(x, dim, stride):
    """x with another stride of its dimension `dim` of extent 1."""
    st = list(x.stride())
    st[dim] = stride
    return torch.as_strided(x, x.shape, st, x.storage_offset())


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,stride", [(1, 6, 2, 5), (1, 4, 4, 0), (7, 1, 1, 3), (7, 1, 1, 0), (1, 1, 1, 1),
                                             (7, 1, 1, (1 << 62) - 1)])
def test_append_and_read_back(quant, dtype, T, Hq, Hkv, stride):
    d, cap = 64, 128
    g = torch.Generator("cuda").manual_seed(T)
    q, k, v = (torch.randn((T, h, d), device="cuda", generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([66 + T], dtype=torch.int32, device="cuda")
    rotary = hils.Rotary(hils.rotary_table(cap, 32))
    shape, kind = ((3, Hkv, C * 40), torch.uint8) if quant else ((3, Hkv, C, d), dtype)

    def run(change):
        kp, vp = (torch.zeros(shape, dtype=kind, device="cuda") for _ in range(2))
        out = hils.kv_append(kp, vp, table, change(k), change(v), lens, rotary=rotary, q=change(q),
                             q_out=change(torch.empty_like(q)))
        got = [kp, vp, out.contiguous()]
        if quant:
            got += [t.contiguous() for t in hils.kv_read(kp, vp, table, lens, T, dtype, k_out=change(torch.empty_like(k)))]
        return got

    dim = 0 if T == 1 else 1
    want, got = run(lambda x: x), run(lambda x: _odd(x, dim, stride) if x.shape[dim] == 1 else x)
    assert hils.hils_get_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
