"""Chunk-paged serving calls: what is refused before any launch (no GPU), and
the 4-bit layout's plain definition against itself."""
import ctypes

import numpy as np
import pytest
import torch

from chunk_wise_sparse_b200 import hils
from tests import paged_reference as ref


@pytest.fixture(scope="module")
def lib():
    from chunk_wise_sparse_b200 import build
    build.build()
    return hils.lib()


P = ctypes.c_void_p(256)      # never dereferenced: validation fails first, or nothing is launched
BAD = ctypes.c_void_p(264)


def dims(**kw):
    base = dict(batch=2, heads_q=4, heads_kv=2, head_dim=64, seqlen=1024, topk=4, dtype=hils.BF16, window=0)
    base.update(kw)
    return hils.make_dims(base["batch"], base["heads_q"], base["heads_kv"], base["head_dim"], base["seqlen"],
                          base["topk"], base["dtype"], base.get("chunk", 64), base["window"])


def tokens(T=6, cu=256, lens=256):
    return ctypes.byref(hils.hils_tokens(T, cu, lens))


def rows(H, data=256, ts=None, hs=64):
    return ctypes.byref(hils.hils_rows(data, H * 64 if ts is None else ts, hs))


def rotary(table=256, n_pos=1024, rot=64, il=0):
    return ctypes.byref(hils.hils_rotary(table, n_pos, rot, il))


def append(lib, d=None, tk=None, ro=None, **kw):
    d = d or dims()
    a = dict(q=rows(4), q_out=rows(4, data=1 << 20), k=rows(2), v=rows(2), kp=P, vp=P, table=P, n=9)
    a.update(kw)
    got = {f(ctypes.byref(d), tk or tokens(), ro, a["q"], a["q_out"], a["k"], a["v"], a["kp"], a["vp"], a["table"],
             a["n"], None) for f in (lib.hils_kv_append_paged, lib.hils_kv_append_quant)}
    assert len(got) == 1
    return got.pop()


@pytest.mark.parametrize("kw,code", [
    (dict(chunk=32), 2), (dict(head_dim=96), 2), (dict(seqlen=1000), 1), (dict(dtype=7), 1), (dict(batch=0), 1),
    (dict(heads_q=3), 1), (dict(topk=0), 2), (dict(window=100), 1),
])
def test_bad_dims(lib, kw, code):
    d = ctypes.byref(dims(**kw))
    assert append(lib, dims(**kw)) == code
    assert lib.hils_kv_read_quant(d, tokens(), P, P, P, 9, rows(2), rows(2), None) == code
    for f in (lib.hils_landmark_summary_append, lib.hils_landmark_summary_quant):
        assert f(d, tokens(), P, P, 9, P, P, P, None, None) == code
    assert lib.hils_attn_decode_quant(d, P, None, P, P, P, 9, P, P, P, P, P, None, None, P, 1 << 40, None) == code
    assert hils.hils_quant_page_bytes(dims(**kw)) == 0 and hils.hils_decode_quant_workspace_bytes(dims(**kw)) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_page_bytes(lib, d):
    n = hils.hils_quant_page_bytes(dims(head_dim=d))
    assert n == 2 * 64 * (d // 2 + d // 8)
    assert hils.quant_pages(3, 2, d, device="cpu").shape == (3, 2, n // 2)


def test_batch_description(lib):
    before = hils.hils_kernel_launches()
    assert append(lib, tk=tokens(-1)) == 1
    assert append(lib, tk=tokens(7, cu=None)) == 1                     # 7 tokens are not shared evenly by 2 sequences
    assert append(lib, tk=tokens(1 << 31)) == 2
    assert append(lib, tk=tokens(6, lens=None)) == 1
    assert append(lib, tk=tokens(6, lens=260)) == 1
    assert append(lib, tk=tokens(6, cu=264)) == 1
    assert lib.hils_kv_append_paged(ctypes.byref(dims()), None, None, None, None, rows(2), rows(2), P, P, P, 9, None) == 1
    # no tokens: nothing is done, whatever the pointers
    none = tokens(0, None, None)
    assert append(lib, tk=none, k=None, v=None, kp=None, vp=None, table=None) == 0
    d = ctypes.byref(dims())
    assert lib.hils_kv_read_quant(d, none, None, None, None, 9, rows(2, data=None), None, None) == 0
    for f in (lib.hils_landmark_summary_append, lib.hils_landmark_summary_quant):
        assert f(d, none, None, None, 9, None, None, None, None, None) == 0
    assert hils.hils_kernel_launches() == before


@pytest.mark.parametrize("ro", [
    rotary(rot=8), rotary(rot=24), rotary(rot=80), rotary(rot=0), rotary(table=None), rotary(table=264),
    rotary(n_pos=0), rotary(il=2),
])
def test_rotary_refused(lib, ro):
    assert append(lib, ro=ro) == 1


@pytest.mark.parametrize("kw", [
    dict(q_out=None), dict(q=None), dict(k=None), dict(v=None), dict(kp=None), dict(vp=BAD), dict(table=None),
    dict(table=BAD), dict(n=0), dict(k=rows(2, data=264)), dict(k=rows(2, ts=129)), dict(k=rows(2, hs=4)),
    dict(v=rows(2, ts=-128)), dict(q_out=rows(4, data=1 << 20, ts=0)), dict(q_out=rows(4, data=1 << 20, hs=0)),
    dict(q_out=rows(4, data=1 << 20, ts=64, hs=64)), dict(q_out=rows(4, data=1 << 20, ts=128, hs=64)),
    dict(k=rows(2, ts=1 << 61)), dict(q_out=rows(4, data=1 << 20, hs=1 << 61)), dict(v=rows(2, hs=1 << 62)),
])
def test_rows_and_pages_refused(lib, kw):
    assert append(lib, **kw) == 1


def test_read_refused(lib):
    d = ctypes.byref(dims())
    ok = rows(2)
    f = lib.hils_kv_read_quant
    assert f(d, tokens(), P, P, P, 9, None, None, None) == 1
    assert f(d, tokens(), None, P, P, 9, ok, ok, None) == 1
    assert f(d, tokens(), P, None, P, 9, ok, ok, None) == 1
    assert f(d, tokens(), P, P, None, 9, ok, ok, None) == 1
    assert f(d, tokens(), P, P, P, 0, ok, ok, None) == 1
    assert f(d, tokens(), P, P, P, 9, rows(2, ts=64), ok, None) == 1      # two heads on the same rows


def test_summary_refused(lib):
    d = ctypes.byref(dims())
    for f in (lib.hils_landmark_summary_append, lib.hils_landmark_summary_quant):
        good = [P, P, 9, P, P, P, P]
        for i in (0, 1, 3, 4, 5):
            assert f(d, tokens(), *[None if j == i else a for j, a in enumerate(good)], None) == 1
        assert f(d, tokens(), P, P, 0, P, P, P, P, None) == 1
        assert f(d, tokens(), P, P, 9, P, P, P, BAD, None) == 1
        # the scoring operand is a bf16 matter
        assert f(ctypes.byref(dims(dtype=hils.FP32)), tokens(), P, P, 9, P, P, P, P, None) == 1


def test_decode_refused(lib):
    d = dims()
    need = hils.hils_decode_quant_workspace_bytes(d)
    assert need > 0
    f = lib.hils_attn_decode_quant
    good = [P, None, P, P, P, 9, None, None, P, P, P, None, None, P, need, None]
    for i in (0, 2, 3, 4, 8, 9, 10, 13):
        assert f(ctypes.byref(d), *[None if j == i else a for j, a in enumerate(good)]) == 1, i
    for i, bad in ((1, BAD), (5, 0), (11, BAD), (12, BAD)):
        assert f(ctypes.byref(d), *[bad if j == i else a for j, a in enumerate(good)]) == 1, i
    assert f(ctypes.byref(d), *[need - 1 if j == 14 else a for j, a in enumerate(good)]) == 4
    big = dims(heads_q=66, heads_kv=2)
    assert f(ctypes.byref(big), *[1 << 40 if j == 14 else a for j, a in enumerate(good)]) == 2
    many = dims(batch=40000)
    assert f(ctypes.byref(many), *[1 << 50 if j == 14 else a for j, a in enumerate(good)]) == 2
    f32 = dims(dtype=hils.FP32)
    assert f(ctypes.byref(f32), *[1 << 40 if j == 14 else a for j, a in enumerate(good)]) == 1     # needs k' and b'


def test_python_layer_refuses(lib):
    """Shapes, types and devices, before the library is called."""
    bf = dict(dtype=torch.bfloat16)
    k = torch.zeros((4, 2, 64), **bf)
    pool, table = torch.zeros((9, 2, 64, 64), **bf), torch.zeros((2, 8), dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    quant = hils.quant_pages(9, 2, 64, device="cpu")
    before = hils.hils_kernel_launches()
    with pytest.raises(ValueError, match="CUDA tensor"):
        hils.kv_append(pool, pool, table, k, k, lens)
    for bad in (dict(seqlens=lens.long()), dict(seqlens=lens[:1]), dict(v=k.float()), dict(k=k[:, :1]),
                dict(page_table=table.long()), dict(cu_tokens=lens), dict(k_pages=pool.float()),
                dict(v_pages=quant), dict(k_pages=quant[..., :100], v_pages=quant[..., :100]),
                dict(q=k[:3]), dict(q_out=k), dict(q=k, q_out=k.float())):
        a = dict(k_pages=pool, v_pages=pool, page_table=table, k=k, v=k, seqlens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            hils.kv_append(**a)
    with pytest.raises(ValueError, match="4-bit"):
        hils.kv_read(pool, pool, table, lens, 4, torch.bfloat16)
    with pytest.raises(ValueError, match="4-bit"):
        hils.decode_step_quant(k[:2], pool, pool, table, None, lens, 4)
    with pytest.raises(ValueError, match="rotary table"):
        hils.Rotary(torch.zeros(4, 16, dtype=torch.float64))
    with pytest.raises(ValueError, match="kprime"):
        hils.landmark_summary_append(quant, table, torch.zeros((2, 2, 8, 64), **bf), lens, 4,
                                     hils.Summary.of(torch.zeros(2, 2, 7, 64), torch.zeros(2, 2, 8)))
    assert hils.hils_kernel_launches() == before


@pytest.mark.parametrize("d", [64, 128])
def test_reference_layout_is_a_bijection_and_pack_inverts(d):
    spots = {ref.unit_and_nibble(i, d) for i in range(d)}
    assert len(spots) == d and {b for b, _ in spots} == set(range(d // 2))
    x = np.random.default_rng(d).standard_normal((3, 2, 64, d))
    codes, step, least = ref.unpack(ref.pack(x), d)
    _, want, s, m = ref.quantise(x)
    assert np.array_equal(codes, want) and np.array_equal(step, s) and np.array_equal(least, m)
    assert np.max(np.abs(ref.values(ref.pack(x), d) - x)) <= 0.52 * s.max()


def test_rotary_table_is_computed_in_64_bits():
    t = hils.rotary_table(1 << 20, 16, device="cpu")
    pos = (1 << 20) - 1
    angle = pos * 10000.0 ** (-np.arange(0, 16, 2) / 16)
    # angles reach 1e6: 64 bits keep them within 1e6 * 2^-53, the table's rounding is 2^-24
    assert np.max(np.abs(t[pos].numpy() - np.concatenate([np.cos(angle), np.sin(angle)]))) <= 2.0 ** -24 + 1e-9
