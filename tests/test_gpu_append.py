"""Appending to a chunk-paged cache with the position rotation, in the cache's
type and in 4 bits, the read-back of 4-bit rows and the summaries of completed
chunks, against plain 64-bit definitions (tests/paged_reference.py).

Tolerances.  A rotated value is x c -+ y s in fp32, two products and a sum of
one rounding each at most (the first product may be fused), then one rounding
to the stored type: eps(t)/2 |result| + 3 * 2^-24 (|x c| + |y s|), with a
quarter more for the products of the roundings.  4-bit rows: see _check_quant.
"""
import numpy as np
import pytest
import torch

from chunk_wise_sparse_b200 import hils
from oracle.oracle import Oracle
from tests import paged_reference as ref
from tests.helpers import SUMMARY_TOL

pytestmark = pytest.mark.gpu

C = 64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _make(dtype, Hq, Hkv, d, seqlens, new, cap, fused=False, pad=0, seed=0, scale=1.0):
    """A ragged batch: packed q, k, v (views of one fused tensor, or dense), seqlens, cu, a page table in no order."""
    g = torch.Generator("cuda").manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) + pad
    x = (torch.randn((T, Hq + 2 * Hkv, d), device="cuda", generator=g) * scale).to(dtype)
    parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    q, k, v = parts if fused else tuple(p.contiguous() for p in parts)
    B, nc = len(seqlens), cap // C
    n_pages = B * nc + 3
    table = torch.randperm(n_pages, device="cuda", generator=g)[: B * nc].to(torch.int32).view(B, nc)
    return dict(q=q, k=k, v=v, T=T, cu=torch.from_numpy(cu).cuda(), cu_host=cu, lens=np.asarray(seqlens, np.int32),
                seqlens=torch.tensor(seqlens, dtype=torch.int32, device="cuda"), table=table, n_pages=n_pages,
                table_host=table.cpu().numpy(), Hkv=Hkv, d=d, dtype=dtype, cap=cap)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _expected(m, table, interleaved, n_pos=None):
    """{(page, row): token} of the tokens that are placed, and rotated q, k with their tolerances."""
    at = ref.places(m["lens"].tolist(), m["cu_host"].tolist())
    pos = np.zeros(m["T"], np.int64)
    for t, _, p in at:
        pos[t] = p
    where = {(int(m["table_host"][b, p // C]), p % C): t for t, b, p in at}
    tab = None if table is None else table.cpu().numpy()
    half = HALF_STEP[m["dtype"]]
    out = {}
    for name in ("q", "k"):
        y, mag = ref.rotate(_f64(m[name]), tab, pos, interleaved)
        out[name] = y, half * np.abs(y) + 1.25 * 3 * 2.0 ** -24 * mag
    return where, out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,Hq,Hkv,rot,interleaved,fused", [
    (64, 4, 2, 64, False, True), (64, 3, 1, 16, True, False), (128, 8, 8, 128, False, False),
    (128, 14, 2, 48, False, True), (128, 5, 5, 128, True, True), (64, 7, 7, 0, False, False), (128, 2, 1, 96, True, True),
])
def test_append_places_and_rotates(dtype, d, Hq, Hkv, rot, interleaved, fused):
    """Ragged: one token, none, a run over several chunks from inside one, a whole prompt; everything else stays."""
    cap = 320
    m = _make(DTYPES[dtype], Hq, Hkv, d, seqlens=[1, 130, 200, 320, 64], new=[1, 0, 139, 320, 2], cap=cap, fused=fused,
              pad=3, seed=d + rot)
    table = hils.rotary_table(cap, rot) if rot else None
    kp = torch.full((m["n_pages"], Hkv, C, d), 7.0, dtype=m["dtype"], device="cuda")
    vp = torch.full_like(kp, -3.0)
    q_out = torch.full((m["T"], Hq, d), 5.0, dtype=m["dtype"], device="cuda")
    rotary = hils.Rotary(table, interleaved) if rot else None
    got = hils.kv_append(kp, vp, m["table"], m["k"], m["v"], m["seqlens"], cu_tokens=m["cu"], rotary=rotary, q=m["q"],
                         q_out=q_out)
    assert got is q_out and hils.hils_get_status() == 0
    where, want = _expected(m, table, interleaved)
    assert len(where) == m["T"] - 3
    pages, rows, toks = (np.array(x) for x in zip(*[(p, r, t) for (p, r), t in where.items()]))
    kg, vg, qg = _f64(kp), _f64(vp), _f64(q_out)
    y, tol = want["k"]
    assert np.all(np.abs(kg[pages, :, rows] - y[toks]) <= tol[toks])
    assert np.array_equal(vg[pages, :, rows], _f64(m["v"])[toks])
    y, tol = want["q"]
    assert np.all(np.abs(qg - y)[:-3] <= tol[:-3])
    assert np.all(qg[-3:] == 5.0)                       # padding behind the last sequence
    kg[pages, :, rows], vg[pages, :, rows] = 7.0, -3.0
    assert np.all(kg == 7.0) and np.all(vg == -3.0)


def test_append_in_place_without_cu_and_head_major():
    """cu_tokens None: the same number of tokens each; q rotated in place; k, v head-major."""
    m = _make(torch.bfloat16, 6, 2, 64, seqlens=[70, 5, 128], new=[5, 5, 5], cap=128, seed=2)
    table = hils.rotary_table(128, 32)
    rotary = hils.Rotary(table)
    kp, vp, kp2, vp2 = (torch.zeros((m["n_pages"], 2, C, 64), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    want = hils.kv_append(kp, vp, m["table"], m["k"], m["v"], m["seqlens"], cu_tokens=m["cu"], rotary=rotary, q=m["q"])
    head_major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (m["q"], m["k"], m["v"])]
    assert not head_major[1].is_contiguous()
    q = head_major[0]
    got = hils.kv_append(kp2, vp2, m["table"], head_major[1], head_major[2], m["seqlens"], rotary=rotary, q=q, q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(kp, kp2) and torch.equal(vp, vp2)
    # without queries the same keys and values
    kp2.zero_(), vp2.zero_()
    assert hils.kv_append(kp2, vp2, m["table"], m["k"], m["v"], m["seqlens"], rotary=rotary) is None
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2)
    # one vector broadcast to all heads and tokens (strides of zero)
    one = torch.randn((1, 1, 64), device="cuda").bfloat16()
    hils.kv_append(kp2, vp2, m["table"], one.expand(15, 2, 64), one.expand(15, 2, 64), m["seqlens"])
    rows = [vp2[int(m["table_host"][b, p // C]), :, p % C] for _, b, p in ref.places(m["lens"].tolist(), m["cu_host"].tolist())]
    assert all(torch.equal(r, one[0].expand(2, 64)) for r in rows)
    assert hils.hils_get_status() == 0


@pytest.mark.parametrize("B", [31, 32, 33, 1024, 1025, 3000])
def test_many_sequences(B):
    """Batches around the steps of the search for a token's sequence, of sequences with no, one or several new tokens:
    every row lands where the plain placing says, in both kinds of page, and is read back from there."""
    rng = np.random.default_rng(B)
    cap, d = 128, 64
    new = rng.integers(0, 3, B)
    new[rng.integers(0, B, 5)] = 40
    lens = np.minimum(cap, new + rng.integers(0, cap, B))
    m = _make(torch.bfloat16, 1, 1, d, seqlens=lens, new=new, cap=cap, seed=B)
    kp, vp = (torch.zeros((m["n_pages"], 1, C, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hils.kv_append(kp, vp, m["table"], m["k"], m["v"], m["seqlens"], cu_tokens=m["cu"])
    at = np.array(ref.places(lens.tolist(), m["cu_host"].tolist()))
    page = torch.from_numpy(m["table_host"][at[:, 1], at[:, 2] // C].astype(np.int64)).cuda()
    row = torch.from_numpy(at[:, 2] % C).cuda()
    want_k, want_v = torch.zeros_like(kp), torch.zeros_like(vp)
    want_k[page, :, row], want_v[page, :, row] = m["k"], m["v"]
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    k4, v4 = hils.quant_pages(m["n_pages"], 1, d), hils.quant_pages(m["n_pages"], 1, d)
    hils.kv_append(k4, v4, m["table"], m["k"], m["v"], m["seqlens"], cu_tokens=m["cu"])
    k, v = hils.kv_read(k4, v4, m["table"], m["seqlens"], m["T"], torch.bfloat16, cu_tokens=m["cu"])
    assert hils.hils_get_status() == 0
    for got, x in ((k, m["k"]), (v, m["v"])):
        x = x.float()
        # half a step of the group's range, the roundings of its ends to fp16 and of the value to bf16
        g = x.view(*x.shape[:2], -1, 32)
        step = (g.amax(-1) - g.amin(-1)) / 15
        tol = (0.5 * step + 2.0 ** -10 * g.abs().amax(-1))[..., None] + 2.0 ** -8 * g.abs() + 2.0 ** -8 * step[..., None]
        assert bool(((got.float().view(g.shape) - g).abs() <= tol).all())
    # one of the two alone
    only = torch.zeros_like(k)
    dims = hils.make_dims(B, 1, 1, d, cap, 1, torch.bfloat16)
    hils.hils_kv_read_quant(dims, m["seqlens"], m["T"], m["cu"], None, v4, m["table"], m["n_pages"], None, only)
    assert torch.equal(only, v) and hils.hils_get_status() == 0


def test_append_far_positions():
    """Positions near the end of a long sequence: offsets of the page pool beyond 2^31 elements, angles of 1e6."""
    d, H, cap = 128, 8, 1 << 20
    n_pages = 40000                               # x 8 x 64 x 128 = 2.6e9 elements
    table = torch.full((2, cap // C), -1, dtype=torch.int32, device="cuda")
    table[0, -1], table[1, -1] = n_pages - 1, n_pages - 2
    rotary = hils.Rotary(hils.rotary_table(cap, d))
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((2, H, d), device="cuda", generator=g).bfloat16() for _ in range(2))
    lens = torch.tensor([cap, cap - 1], dtype=torch.int32, device="cuda")
    kp = torch.empty((n_pages, H, C, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    hils.kv_append(kp, vp, table, k, v, lens, rotary=rotary)
    assert hils.hils_get_status() == 0
    y, mag = ref.rotate(_f64(k), rotary.table.cpu().numpy(), np.array([cap - 1, cap - 2]), False)
    tol = 2.0 ** -8 * np.abs(y) + 1.25 * 3 * 2.0 ** -24 * mag
    for b, (page, row) in enumerate([(n_pages - 1, 63), (n_pages - 2, 62)]):
        assert np.all(np.abs(_f64(kp[page, :, row]) - y[b]) <= tol[b])
        assert torch.equal(vp[page, :, row], v[b])


@pytest.mark.parametrize("quant", [False, True])
def test_append_records_what_does_not_fit_and_skips_it(quant):
    """A sequence longer than the cache, one shorter than its new tokens, a page outside the pool, a position outside
    the rotary table: recorded; the sequences that fit are written as without them."""
    def pools():
        if quant:
            return [torch.full((m["n_pages"], 2, C * 40), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
        return [torch.full((m["n_pages"], 2, C, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    m = _make(torch.bfloat16, 4, 2, 64, seqlens=[10, 66, 128, 70], new=[3, 2, 5, 6], cap=128, seed=4)
    rotary = hils.Rotary(hils.rotary_table(128, 64))
    kp, vp = pools()
    want_q = hils.kv_append(kp, vp, m["table"], m["k"], m["v"], m["seqlens"], cu_tokens=m["cu"], rotary=rotary, q=m["q"])
    assert hils.hils_get_status() == 0
    for case in ("long", "short", "page", "table", "negative"):
        lens, table, rot = m["lens"].copy(), m["table"].clone(), rotary
        bad = 2
        if case == "long":
            lens[bad] = 129
        elif case == "short":
            lens[bad] = 4
        elif case == "negative":
            lens[bad] = -7
        elif case == "page":
            table[bad, 1] = m["n_pages"]
        else:
            rot = hils.Rotary(rotary.table[:100].contiguous())          # only sequence 2 reaches position 100
        kp2, vp2 = pools()
        q2 = torch.full_like(want_q, 3.0)
        hils.kv_append(kp2, vp2, table, m["k"], m["v"], torch.from_numpy(lens).cuda(), cu_tokens=m["cu"], rotary=rot,
                       q=m["q"], q_out=q2)
        assert hils.hils_get_status() == 6, case
        keep = np.ones(m["T"], bool)
        keep[5:10] = False
        assert torch.equal(q2[keep], want_q[keep])
        assert torch.equal(q2[5:10], want_q[5:10]) if case == "page" else bool((q2[5:10] == 3).all()), case
        for a, b in ((kp, kp2), (vp, vp2)):
            touched = (a != b).flatten(1).any(1).nonzero().flatten().tolist()
            assert touched == [int(m["table_host"][bad, 1])], case       # its rows alone are missing
    # cu_tokens beyond the packed tokens, and not ascending
    for cu in ([0, 3, 5, 10, 17], [0, 3, 2, 10, 16]):
        kp2, vp2 = pools()
        hils.kv_append(kp2, vp2, m["table"], m["k"], m["v"], m["seqlens"],
                       cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"), rotary=rotary, q=m["q"])
        assert hils.hils_get_status() == 6
    # a negative page, and a whole table of pages outside the pool
    kp2, vp2 = pools()
    hils.kv_append(kp2, vp2, torch.full_like(m["table"], -1), m["k"], m["v"], m["seqlens"], cu_tokens=m["cu"])
    assert hils.hils_get_status() == 6
    assert all(torch.equal(a, b) for a, b in zip((kp2, vp2), pools()))


def _check_quant(pages, x, noise, where, H, d, exact):
    """The rows of `pages` that `where` names against x [T, H, d] in 64 bits, each known to `noise`.

    m is fp16(min): within 2^-11 |min| + 2^-25 (half a subnormal step) + noise.  s: the same of (max - min) / 15, with
    2 noise / 15 and a division's 2^-24.  A value takes the nearest code, so it is off by s / 2, or, at the two ends,
    by what the roundings of m and of 15 s leave outside: |m - min| and 15 |s - (max - min)/15|.  `exact`: the inputs
    were exact, so the codes are the plain ones of the stored s and m, except within 1e-5 of half way between two (x - m
    and the quotient carry 2^-24 of at most 16 each: 2e-6).  s and m themselves: max - min and its 15th carry 2^-24 each
    in fp32, so the rounding to fp16 falls on the other side only within 2^-23 of half way between two fp16 values: on
    at most 2^-23 / 2^-11 of the groups, and the difference of two bf16 values of like size is exact."""
    codes, step, least = ref.unpack(pages, d)
    pg, rw, tk = (np.array(v) for v in zip(*[(p, r, t) for (p, r), t in where.items()]))
    codes, step, least = codes[pg, :, rw], step[pg, :, rw], least[pg, :, rw]
    y, n = x[tk], noise[tk]
    g = y.reshape(len(tk), H, -1, 32)
    n_g = n.reshape(g.shape).max(-1)
    lo, hi = g.min(-1), g.max(-1)
    tol_m = 2.0 ** -11 * (np.abs(lo) + n_g) + 2.0 ** -25 + n_g
    tol_s = (2.0 ** -11 + 2.0 ** -22) * ((hi - lo) + 2 * n_g) / 15 + 2.0 ** -25 + 2 * n_g / 15
    assert np.all(np.abs(least - lo) <= tol_m)
    assert np.all(np.abs(step - (hi - lo) / 15) <= tol_s)
    held = (least[..., None] + step[..., None] * codes.reshape(g.shape))
    bound = np.maximum(step / 2 * (1 + 2.0 ** -20), tol_m + 15 * tol_s)[..., None] + n.reshape(g.shape)
    assert np.all(np.abs(held - g) <= bound)
    if exact:
        _, _, s, m = ref.quantise(y)
        assert np.array_equal(least, m) and np.mean(step != s) <= 8 * 2.0 ** -12
        with np.errstate(divide="ignore", invalid="ignore"):
            ratio = np.where(step[..., None] > 0, (g - least[..., None]) / step[..., None], 0.0).reshape(y.shape)
        want = np.clip(np.rint(ratio), 0, 15)
        near_half = np.abs(ratio - np.floor(ratio) - 0.5) < 1e-5
        assert np.all((codes == want) | near_half)
        assert np.mean(codes != want) <= 1e-4
    return codes


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,Hq,Hkv,rot,interleaved,fused,queries", [
    (64, 4, 2, 64, False, True, True), (128, 8, 8, 128, True, False, True), (128, 14, 2, 48, False, True, True),
    (64, 1, 1, 0, False, False, False), (128, 3, 3, 32, False, False, True),
])
def test_append_in_4_bits(dtype, d, Hq, Hkv, rot, interleaved, fused, queries):
    cap = 320
    m = _make(DTYPES[dtype], Hq, Hkv, d, seqlens=[1, 130, 200, 320, 64], new=[1, 0, 139, 320, 2], cap=cap, fused=fused,
              pad=2, seed=d + rot)
    table = hils.rotary_table(cap, rot) if rot else None
    nb = C * (d // 2 + d // 8)
    kp, vp = (torch.full((m["n_pages"], Hkv, nb), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    kw = dict(cu_tokens=m["cu"], rotary=hils.Rotary(table, interleaved) if rot else None)
    q = hils.kv_append(kp, vp, m["table"], m["k"], m["v"], m["seqlens"], q=m["q"] if queries else None, **kw)
    assert hils.hils_get_status() == 0
    where, want = _expected(m, table, interleaved)
    if queries:
        y, tol = want["q"]
        assert np.all(np.abs(_f64(q) - y)[:-2] <= tol[:-2])
    y, _ = want["k"]
    _, mag = ref.rotate(_f64(m["k"]), None if table is None else table.cpu().numpy(), _positions(m), interleaved)
    _check_quant(kp.cpu().numpy(), y, 1.25 * 3 * 2.0 ** -24 * mag, where, Hkv, d, exact=rot == 0)
    v = _f64(m["v"])
    _check_quant(vp.cpu().numpy(), v, np.zeros_like(v), where, Hkv, d, exact=True)
    # everything else stays
    for pages in (kp, vp):
        left = pages.cpu().numpy()
        codes = left[:, :, : C * d // 2].reshape(m["n_pages"], Hkv, C, -1)
        pars = left[:, :, C * d // 2:].reshape(m["n_pages"], Hkv, C, -1)
        for p, r in where:
            codes[p, :, r], pars[p, :, r] = 0xA5, 0xA5
        assert np.all(codes == 0xA5) and np.all(pars == 0xA5)
    # read back: m + s * code, rounded to fp32 once and then to the type
    k2, v2 = hils.kv_read(kp, vp, m["table"], m["seqlens"], m["T"], m["dtype"], cu_tokens=m["cu"],
                          k_out=torch.full_like(m["k"].contiguous(), 2.0))
    assert hils.hils_get_status() == 0
    assert bool((k2[-2:] == 2.0).all())
    for pages, got in ((kp, k2), (vp, v2)):
        held = torch.from_numpy(ref.values(pages.cpu().numpy(), d))
        for (p, r), t in where.items():
            assert torch.equal(got[t].cpu(), held[p, :, r].to(m["dtype"]))


def _positions(m):
    pos = np.zeros(m["T"], np.int64)
    for t, _, p in ref.places(m["lens"].tolist(), m["cu_host"].tolist()):
        pos[t] = p
    return pos


def test_4_bit_edges():
    """Groups of one value, of zeros, far from zero, tiny, of both signs; infinities, NaN and values beyond fp16 make
    their group NaN and no other."""
    d, H = 64, 1
    x = torch.zeros((12, H, d), device="cuda")
    x[1] = 3.25
    x[2, :, ::2] = -1e-3
    x[3] = torch.linspace(1000, 1001, d, device="cuda")
    x[4] = torch.linspace(-1e-7, 1e-7, d, device="cuda")           # the step is a subnormal of fp16
    x[5, :, 5] = float("inf")
    x[6, :, 40] = float("-inf")
    x[7, :, 0] = float("nan")
    x[8, :, 33] = 70000.0                                          # the step fits fp16 (4667), so does the least
    x[9, :, 1] = -70000.0                                          # the least value does not
    x[10, :, 2] = 1e30
    x[11] = torch.where(torch.arange(d, device="cuda") % 2 == 0, 60000.0, -60000.0)
    table = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([12], dtype=torch.int32, device="cuda")
    kp, vp = hils.quant_pages(3, H, d), hils.quant_pages(3, H, d)
    hils.kv_append(kp, vp, table, x, x, lens)
    k, v = hils.kv_read(kp, vp, table, lens, 12, torch.float32)
    assert hils.hils_get_status() == 0 and torch.equal(kp, vp)
    assert torch.equal(torch.nan_to_num(k, 123.0), torch.nan_to_num(v, 123.0))
    k = k[:, 0].cpu()
    assert bool((k[0] == 0).all()) and bool((k[1] == 3.25).all())
    nan = torch.isnan(k).view(12, 2, 32)
    want = torch.zeros((12, 2), dtype=torch.bool)
    for row, group in ((5, 0), (6, 1), (7, 0), (9, 0), (10, 0)):
        want[row, group] = True
    assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)
    y = x[:, 0].cpu()
    # half a step of the group's range and the rounding of its ends to fp16 (2^-11 of them, 2^-25 below its range)
    lo, hi = y.view(12, 2, 32).amin(-1), y.view(12, 2, 32).amax(-1)
    tol = (hi - lo) / 30 * (1 + 2.0 ** -10) + 2.0 ** -10 * torch.maximum(lo.abs(), hi.abs()) + 16 * 2.0 ** -25
    err = (k - y).abs().view(12, 2, 32).amax(-1)
    assert bool((err[~want] <= tol[~want]).all())


@pytest.mark.parametrize("dtype,quant,d,H", [("bf16", True, 64, 2), ("bf16", True, 128, 3), ("fp32", True, 64, 1),
                                             ("fp32", True, 128, 2), ("bf16", False, 64, 3), ("bf16", False, 128, 2),
                                             ("fp32", False, 64, 2), ("fp32", False, 128, 1)])
@pytest.mark.parametrize("lens,new", [
    ([1, 64, 200, 320, 191], [1, 64, 139, 320, 0]),       # a first token, exactly a chunk, several, all, none
    ([64, 128, 192, 63], [1, 1, 1, 1]),                   # single tokens: three complete a chunk, one does not
    ([320], [5]), ([127], [127]),
])
def test_summaries_of_completed_chunks(dtype, quant, d, H, lens, new):
    cap, B = 320, len(lens)
    nc = cap // C
    rng = np.random.default_rng(d + H)
    g = torch.Generator("cuda").manual_seed(d)
    dt = DTYPES[dtype]
    n_pages = B * nc + 2
    table = torch.randperm(n_pages, device="cuda", generator=g)[: B * nc].to(torch.int32).view(B, nc)
    x = rng.standard_normal((n_pages, H, C, d)).astype(np.float32)
    if quant:
        pages = torch.from_numpy(ref.pack(x)).cuda()
        dense = ref.values(pages.cpu().numpy(), d)
    else:
        pages = torch.from_numpy(x).to(dt).cuda()
        dense = pages.float().cpu().numpy()
    lq = torch.randn((B, H, nc, d), device="cuda", generator=g).to(dt)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    dims = hils.make_dims(B, H, H, d, cap, 1, dt)
    summ = hils.Summary(dims, "cuda")
    bufs = [t for t in (summ.kprime, summ.bprime, summ.kprime_mma) if t is not None]
    for t in bufs:
        t.fill_(11.0)
    hils.landmark_summary_append(pages, table, lq, torch.tensor(lens, dtype=torch.int32, device="cuda"), int(cu[-1]),
                                 summ, cu_tokens=torch.from_numpy(cu).cuda())
    assert hils.hils_get_status() == 0
    t_host = table.cpu().numpy()
    cache = dense[t_host.reshape(-1)].reshape(B, nc, H, C, d).transpose(0, 2, 1, 3, 4).reshape(B, H, cap, d)
    kp, bp = Oracle(B, H, H, cap, d, C, 1).summary(cache, lq.float().cpu().numpy())
    done = np.zeros((B, nc), bool)
    for b in range(B):
        done[b, (lens[b] - new[b]) // C: lens[b] // C] = True
    sel = np.repeat(done[:, None], H, 1)
    kg, bg = summ.kprime.cpu().numpy(), summ.bprime.cpu().numpy()
    assert np.all(kg[~sel] == 11.0) and np.all(bg[~sel] == 11.0)
    if sel.any():
        assert np.max(np.abs(kg[sel] - kp[sel])) <= SUMMARY_TOL and np.max(np.abs(bg[sel] - bp[sel])) <= SUMMARY_TOL
    if dtype == "bf16":
        mma = summ.kprime_mma.view(B, H, nc, d + 16).cpu()
        pick = torch.from_numpy(sel)
        assert bool((mma[~pick] == 11.0).all())
        assert torch.equal(mma[pick][:, :d], summ.kprime.cpu()[pick].bfloat16())
        # b'/tau as a sum of two bf16 values: the second's rounding is 2^-8 of the first's, 2^-9 each
        x = mma[pick][:, d].double() + mma[pick][:, d + 1].double()
        want = summ.bprime.cpu()[pick].double() * np.sqrt(d)
        assert bool(((x - want).abs() <= 2.0 ** -16 * want.abs() + 1e-5).all())
        assert bool((mma[pick][:, d + 2:] == 0).all())


def test_summary_equals_the_range_call_and_records_a_bad_page():
    """On the cache's own type: what hils_landmark_summary_paged computes for the same chunks; a completed chunk
    without a page is recorded and stays unwritten."""
    B, H, d, cap = 2, 2, 128, 512
    nc = cap // C
    pages = torch.randn((B * nc, H, C, d), device="cuda").bfloat16()
    table = torch.randperm(B * nc, device="cuda").to(torch.int32).view(B, nc)
    lq = torch.randn((B, H, nc, d), device="cuda").bfloat16()
    dims = hils.make_dims(B, H, H, d, cap, 1, torch.bfloat16)
    want, got = hils.Summary(dims, "cuda"), hils.Summary(dims, "cuda")
    hils.hils_landmark_summary_paged(dims, pages, table, B * nc, lq, 0, nc, want.kprime, want.bprime, want.kprime_mma)
    lens = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    hils.landmark_summary_append(pages, table, lq, lens, B * cap, got)
    assert hils.hils_get_status() == 0
    assert (want.kprime - got.kprime).abs().max().item() <= SUMMARY_TOL
    assert (want.bprime - got.bprime).abs().max().item() <= SUMMARY_TOL
    bad = table.clone()
    bad[1, 3] = -5
    got.kprime.fill_(11.0)
    hils.landmark_summary_append(pages, bad, lq, lens, B * cap, got)
    assert hils.hils_get_status() == 6
    assert bool((got.kprime[1, :, 3] == 11.0).all())
    got.kprime[1, :, 3] = want.kprime[1, :, 3]
    assert (want.kprime - got.kprime).abs().max().item() <= SUMMARY_TOL
