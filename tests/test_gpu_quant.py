"""The decode step over a 4-bit chunk-paged cache against the fp64 oracle on
the values that the codes stand for, and the serving loop (append, summaries of
completed chunks, decode) as it is used: ragged, captured in a graph, on a
stream of its own.  Tolerances are those of the other decode tests."""
import numpy as np
import pytest
import torch

from chunk_wise_sparse_b200 import hils
from oracle.oracle import Oracle
from tests import paged_reference as ref
from tests.helpers import OUT_MAX, OUT_MEAN, SEL_GAP, check_selection

pytestmark = pytest.mark.gpu

C = 64
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _cache(B, Hq, Hkv, d, cap, dtype, seed, spread=1.0):
    """A random 4-bit cache with its summaries and a query; `dense`: the values it stands for, [B,Hkv,cap,d]."""
    rng = np.random.default_rng(seed)
    nc, n_pages = cap // C, B * (cap // C) + 4
    table = rng.permutation(n_pages)[: B * nc].astype(np.int32).reshape(B, nc)
    pools, dense = [], []
    for _ in range(2):
        p = ref.pack(rng.standard_normal((n_pages, Hkv, C, d)).astype(np.float32) * spread)
        val = ref.values(p, d)
        dense.append(np.ascontiguousarray(val[table.reshape(-1)].reshape(B, nc, Hkv, C, d).transpose(0, 2, 1, 3, 4)
                                          .reshape(B, Hkv, cap, d)))
        pools.append(torch.from_numpy(p).cuda())
    dt = DTYPES[dtype]
    q = torch.from_numpy(rng.standard_normal((B, Hq, d)).astype(np.float32)).to(dt).cuda()
    lq = torch.from_numpy(rng.standard_normal((B, Hkv, nc, d)).astype(np.float32)).to(dt).cuda()
    tab = torch.from_numpy(table).cuda()
    summ = hils.Summary(hils.make_dims(B, Hkv, Hkv, d, cap, 1, dt), "cuda")
    full = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    hils.landmark_summary_append(pools[0], tab, lq, full, B * cap, summ)
    assert hils.hils_get_status() == 0
    return dict(q=q, lq=lq, kp=pools[0], vp=pools[1], table=tab, table_host=table, n_pages=n_pages, summ=summ,
                k=dense[0], v=dense[1], B=B, Hq=Hq, Hkv=Hkv, d=d, cap=cap, dtype=dtype)


def _against_oracle(m, lens, K, window, got, q_score=None):
    o, ids, scores = got
    oracle = Oracle(m["B"], m["Hq"], m["Hkv"], m["cap"], m["d"], C, K, window)
    kp, bp = oracle.summary(m["k"], m["lq"].float().cpu().numpy())
    q = m["q"].float().cpu().numpy()
    from oracle.oracle import Rows
    rows = Rows.from_decode(q, lens)
    srows = rows if q_score is None else Rows.from_decode(q_score.float().cpu().numpy(), lens)
    want_ids, want_scores, gap = oracle.select(kp, bp, srows)
    ids_g = ids.reshape(-1, K).cpu().numpy()
    tol = SEL_GAP[m["dtype"]]
    check_selection(ids_g, want_ids, gap, oracle.scores(kp, bp, srows), tol, tol)
    O, _ = oracle.attend(m["k"], m["v"], kp, bp, rows, ids_g, qscore=None if q_score is None else srows.q)
    err = np.abs(o.float().reshape(-1, m["d"]).cpu().numpy() - O)
    assert err.max() <= OUT_MAX[m["dtype"]], err.max()
    assert err.mean() <= OUT_MEAN[m["dtype"]], err.mean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hq,Hkv,d,cap,K,window,lens", [
    (1, 1, 1, 64, 64, 1, 0, [1]),                                   # one cached token
    (3, 8, 2, 128, 4096, 16, 0, [4096, 4051, 700]),
    (3, 8, 2, 64, 4096, 16, 512, [4096, 3969, 65]),
    (2, 12, 4, 128, 2048, 3, 0, [2048, 1985]),                      # three heads per kv head
    (4, 7, 1, 64, 1024, 8, 128, [1, 64, 65, 129]),                  # seven, short sequences
    (2, 16, 1, 128, 1024, 4, 0, [1000, 999]),                       # sixteen
    (1, 32, 1, 64, 2048, 5, 64, [2000]),                            # thirty-two
    (2, 20, 2, 64, 1024, 7, 1024, [1024, 1023]),                    # ten; the window covers everything
    (2, 2, 2, 128, 8192, 64, 0, [8192, 6000]),                      # the largest K
    (2, 9, 1, 128, 8192, 64, 192, [8192, 5001]),
    (1, 4, 4, 64, 1 << 19, 16, 0, [(1 << 19) - 3]),                 # 8192 candidates
])
def test_decode_matches_the_oracle(dtype, B, Hq, Hkv, d, cap, K, window, lens):
    m = _cache(B, Hq, Hkv, d, cap, dtype, seed=Hq + d)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, K, window=window, with_selection=True)
    assert hils.hils_get_status() == 0
    _against_oracle(m, np.array(lens), K, window, got)


def test_decode_more_candidates_than_registers_hold():
    """Beyond 8192 candidate chunks the top-K reads its scores from memory again."""
    m = _cache(1, 2, 1, 64, 64 * 9000, "bf16", seed=5)
    lens = np.array([64 * 9000 - 17])
    got = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"],
                                 torch.from_numpy(lens.astype(np.int32)).cuda(), 32, with_selection=True)
    assert hils.hils_get_status() == 0
    _against_oracle(m, lens, 32, 0, got)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_equals_the_unquantised_step_on_the_values_read_back(dtype):
    """kv_read into a contiguous cache, then hils_attn_decode: the same selection, outputs within rounding."""
    m = _cache(2, 8, 2, 128, 2048, dtype, seed=8)
    dt, cap = DTYPES[dtype], m["cap"]
    kc, vc = (torch.empty((2, 2, cap, 128), dtype=dt, device="cuda") for _ in range(2))
    full = torch.tensor([cap], dtype=torch.int32, device="cuda")
    for b in range(2):      # a sequence at a time: rows [T, Hkv, d] that are a view of the head-major cache
        hils.kv_read(m["kp"], m["vp"], m["table"][b:b + 1], full, cap, dt, k_out=kc[b].transpose(0, 1),
                     v_out=vc[b].transpose(0, 1))
    assert np.array_equal(kc.float().cpu().numpy(), torch.from_numpy(m["k"]).to(dt).float().numpy())
    assert np.array_equal(vc.float().cpu().numpy(), torch.from_numpy(m["v"]).to(dt).float().numpy())
    seq = torch.tensor([cap, 1500], dtype=torch.int32, device="cuda")
    o, ids, sc = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 16, with_selection=True)
    o2, ids2, sc2 = hils.decode_step(m["q"], kc, vc, m["summ"], seq, 16)
    assert hils.hils_get_status() == 0
    assert torch.equal(ids, ids2) and (sc - sc2).abs().max().item() <= 1e-5
    assert (o.float() - o2.float()).abs().max().item() <= OUT_MAX[dtype]


def test_decode_with_a_scoring_query_and_without_optional_outputs():
    m = _cache(2, 8, 2, 64, 2048, "bf16", seed=9)
    lens = np.array([2048, 1300])
    seq = torch.from_numpy(lens.astype(np.int32)).cuda()
    qs = torch.randn((2, 8, 64), device="cuda").bfloat16()
    got = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 8, q_score=qs, with_selection=True)
    assert hils.hils_get_status() == 0
    _against_oracle(m, lens, 8, 0, got, q_score=qs)
    dims = hils.make_dims(2, 8, 2, 64, 2048, 8, torch.bfloat16)
    ws = torch.empty((hils.hils_decode_quant_workspace_bytes(dims),), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(m["q"])
    hils.hils_attn_decode_quant(dims, m["q"], qs, m["kp"], m["vp"], m["table"], m["n_pages"], None, None,
                                m["summ"].kprime_mma, seq, o, None, None, ws)
    assert torch.equal(o, got[0])
    o2, ids, sc = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 8, q_score=qs)
    assert torch.equal(o2, o) and ids is None and sc is None


def test_rows_behind_the_sequence_are_not_looked_at():
    """Codes and parameters of positions from seqlens on (here NaN) do not reach the output; a NaN inside does."""
    m = _cache(2, 4, 2, 64, 512, "bf16", seed=10)
    lens = [300, 257]
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    run = lambda: hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 4, window=128)  # noqa: E731
    want = run()[0].clone()
    for pages in (m["kp"], m["vp"]):
        for b, n in enumerate(lens):
            page = pages[int(m["table_host"][b, n // C])]
            page[:, C * 32:].view(2, C, 8)[:, n % C:] = 0xFF       # fp16 NaN
            page[:, : C * 32].view(2, C, 32)[:, n % C:] = 0xFF
            pages[m["table"][b, n // C + 1:].long()] = 0xFF
    got = run()[0]
    assert hils.hils_get_status() == 0
    assert torch.equal(got, want) and bool(torch.isfinite(got.float()).all())
    page = m["vp"][int(m["table_host"][1, 256 // C])]
    page[1, C * 32:].view(C, 8)[0, :4] = 0xFF                      # sequence 1, kv head 1, dims 0 .. 31
    got = run()[0]
    bad = torch.isnan(got.float())
    assert bool(bad[1, 2:, :32].all())
    bad[1, 2:, :32] = False
    assert not bool(bad.any())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_in_a_key_reaches_the_heads_that_read_it(dtype):
    """A group of a cached key that stands for NaN makes its chunk's summary and scores NaN: they sort first, and the
    kv head's query heads become NaN; the other kv head and the other sequence do not change."""
    m = _cache(2, 6, 2, 64, 2048, dtype, seed=13)
    seq = torch.tensor([2048, 2000], dtype=torch.int32, device="cuda")
    args = (m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 8)
    want = hils.decode_step_quant(*args, window=128)[0].clone()
    page = m["kp"][int(m["table_host"][0, 3])]
    page[1, C * 32:].view(C, 8)[5, 4:] = 0xFF                      # sequence 0, kv head 1, chunk 3, key 5, dims 32 .. 63
    full = torch.full((2,), 2048, dtype=torch.int32, device="cuda")
    hils.landmark_summary_append(m["kp"], m["table"], m["lq"], full, 2 * 2048, m["summ"])
    got, ids, _ = hils.decode_step_quant(*args, window=128, with_selection=True)
    assert hils.hils_get_status() == 0
    assert bool(torch.isnan(m["summ"].kprime[0, 1, 3]).all()) and bool((ids[0, 3:] == 3).any(-1).all())
    assert bool(torch.isnan(got[0, 3:].float()).all())
    assert torch.equal(got[0, :3], want[0, :3]) and torch.equal(got[1], want[1])


def test_decode_records_bad_pages_and_lengths():
    m = _cache(3, 4, 2, 64, 1024, "bf16", seed=11)
    seq = torch.tensor([1024, 1000, 900], dtype=torch.int32, device="cuda")
    want, ids, _ = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 4, with_selection=True)
    bad = m["table"].clone()
    bad[1, int(ids[1, 0, 0])] = m["n_pages"]
    o, ids2, _ = hils.decode_step_quant(m["q"], m["kp"], m["vp"], bad, m["summ"], seq, 4, with_selection=True)
    assert hils.hils_get_status() == 6
    assert torch.equal(ids, ids2) and torch.equal(o[[0, 2]], want[[0, 2]]) and bool(torch.isfinite(o.float()).all())
    assert not torch.equal(o[1, 0], want[1, 0])
    bad = m["table"].clone()
    bad[:] = -1                                   # no page at all: nothing is attended
    o, _, _ = hils.decode_step_quant(m["q"], m["kp"], m["vp"], bad, m["summ"], seq, 4)
    assert hils.hils_get_status() == 6 and bool((o == 0).all())
    for n in (0, -1, 1025):
        seq2 = torch.tensor([1024, n, 900], dtype=torch.int32, device="cuda")
        o, ids2, sc = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq2, 4,
                                             with_selection=True)
        assert hils.hils_get_status() == 6
        assert torch.equal(o[[0, 2]], want[[0, 2]]) and bool((o[1] == 0).all()) and bool((ids2[1] == -1).all())
        assert bool((sc[1] == float("-inf")).all())


def test_large_logits_and_equal_rows():
    """Keys and queries whose logits reach thousands; a chunk of equal keys; ties among chunks go to the lower ids."""
    m = _cache(1, 4, 2, 64, 1024, "fp32", seed=12, spread=30.0)
    m["q"].mul_(20)
    lens = np.array([1024])
    seq = torch.tensor([1024], dtype=torch.int32, device="cuda")
    o, ids, _ = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 4, window=128, with_selection=True)
    assert hils.hils_get_status() == 0
    oracle = Oracle(1, 4, 2, 1024, 64, C, 4, 128)
    kp, bp = oracle.summary(m["k"], m["lq"].cpu().numpy())
    from oracle.oracle import Rows
    O, _ = oracle.attend(m["k"], m["v"], kp, bp, Rows.from_decode(m["q"].cpu().numpy(), lens), ids.reshape(-1, 4).cpu().numpy())
    # logits of up to |q||k|/8 = 2e4 carry 2^-24 of themselves and of their terms: the weights are off by up to 1e-2
    # where the two largest are close, and the outputs (|v| up to 1e2) by that share of a difference of values
    assert np.max(np.abs(o.cpu().numpy().reshape(-1, 64) - O)) <= 2e-2 * np.abs(m["v"]).max()
    # every chunk the same page: all scores equal, all outputs the mean of equal branches
    same = torch.zeros_like(m["table"])
    m["summ"].kprime[:] = m["summ"].kprime[:, :, :1].clone()
    m["summ"].bprime[:] = m["summ"].bprime[:, :, :1].clone()
    _, ids, _ = hils.decode_step_quant(m["q"], m["kp"], m["vp"], same, m["summ"], seq, 4, with_selection=True)
    assert ids.view(4, 4).tolist() == [[0, 1, 2, 3]] * 4


@pytest.mark.parametrize("cap", [64 * 700, 64 * 3000, 64 * 33000])
def test_tied_scores_go_to_the_lower_ids(cap):
    """More equal scores than a row's threads: the K kept ones are those above the tie and then the lowest ids of it
    (the row in registers of 256 or 1024 threads, and beyond what registers hold)."""
    K, nc = 16, cap // C
    kp, vp = hils.quant_pages(1, 1, 64), hils.quant_pages(1, 1, 64)
    table = torch.zeros((1, nc), dtype=torch.int32, device="cuda")      # every chunk is the one page
    q = torch.ones((1, 2, 64), device="cuda")
    bias = torch.zeros((1, 1, nc), device="cuda")
    above = [5, 300, 301, nc - 2]
    bias[0, 0, above] = 1.0
    bias[0, 0, 7:20] = -1.0
    bias[0, 0, 2] = float("-inf")
    summ = hils.Summary.of(torch.zeros((1, 1, nc, 64), device="cuda"), bias)
    seq = torch.tensor([cap], dtype=torch.int32, device="cuda")
    _, ids, sc = hils.decode_step_quant(q, kp, vp, table, summ, seq, K, with_selection=True)
    assert hils.hils_get_status() == 0
    tied = [c for c in range(nc - 1) if c not in above and not 7 <= c < 20 and c != 2]
    want = sorted(above + tied[: K - len(above)])
    assert ids.view(2, K).tolist() == [want] * 2
    assert sc.view(2, K).tolist() == [[1.0 if c in above else 0.0 for c in want]] * 2


class _Loop:
    """A serving loop over a ragged batch: its buffers, and one step for one new token of every sequence."""

    def __init__(self, quant, B=3, Hq=8, Hkv=2, d=64, cap=512, K=4, seed=20):
        g = torch.Generator("cuda").manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.d, self.cap, self.K, self.quant = B, Hq, Hkv, d, cap, K, quant
        nc, n_pages = cap // C, B * cap // C + 2
        self.table = torch.randperm(n_pages, device="cuda", generator=g)[: B * nc].to(torch.int32).view(B, nc)
        if quant:
            self.kp, self.vp = hils.quant_pages(n_pages, Hkv, d), hils.quant_pages(n_pages, Hkv, d)
        else:
            self.kp, self.vp = (torch.zeros((n_pages, Hkv, C, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.n_pages = n_pages
        self.x = torch.randn((B, cap, Hq + 2 * Hkv, d), device="cuda", generator=g).bfloat16()     # every token's q, k, v
        self.lq = torch.randn((B, Hkv, nc, d), device="cuda", generator=g).bfloat16()
        self.rotary = hils.Rotary(hils.rotary_table(cap, 32))
        self.dims = hils.make_dims(B, Hq, Hkv, d, cap, K, torch.bfloat16)
        self.summ = hils.Summary(self.dims, "cuda")
        for t in (self.summ.kprime, self.summ.bprime, self.summ.kprime_mma):
            t.zero_()
        self.seqlens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.new = torch.empty((B, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
        need = hils.hils_decode_quant_workspace_bytes if quant else hils.hils_decode_workspace_bytes
        self.ws = torch.empty((need(self.dims),), dtype=torch.uint8, device="cuda")
        self.o = torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda")

    def _split(self, x):
        return x[:, : self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def prompt(self, lens, stream=None):
        x = torch.cat([self.x[b, :n] for b, n in enumerate(lens)])
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        self.seqlens.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        q, k, v = self._split(x)
        hils.kv_append(self.kp, self.vp, self.table, k, v, self.seqlens, cu_tokens=cu, rotary=self.rotary, q=q, stream=stream)
        hils.landmark_summary_append(self.kp, self.table, self.lq, self.seqlens, x.shape[0], self.summ, cu_tokens=cu,
                                     stream=stream)
        self.lens = list(lens)

    def feed(self):
        self.new.copy_(torch.stack([self.x[b, n] for b, n in enumerate(self.lens)]))
        self.lens = [n + 1 for n in self.lens]

    def step(self, stream=None):
        """The device work of one step: everything it needs is in the loop's buffers."""
        self.seqlens.add_(1)
        q, k, v = self._split(self.new)
        q = hils.kv_append(self.kp, self.vp, self.table, k, v, self.seqlens, rotary=self.rotary, q=q, stream=stream)
        hils.landmark_summary_append(self.kp, self.table, self.lq, self.seqlens, self.B, self.summ, stream=stream)
        if self.quant:
            hils.decode_step_quant(q, self.kp, self.vp, self.table, self.summ, self.seqlens, self.K, workspace=self.ws,
                                   out=self.o, stream=stream)
        else:
            hils.hils_attn_decode_paged(self.dims, q, self.kp, self.vp, self.table, self.n_pages, self.summ.kprime,
                                        self.summ.bprime, self.summ.kprime_mma, self.seqlens, self.o, None, None,
                                        self.ws, stream=stream)

    def reference(self):
        """O of the newest tokens from the cache's own values: rotation and cache rebuilt in 64 bits."""
        tab = self.rotary.table.cpu().numpy()
        host = self.x.float().cpu().numpy()
        K, V = (np.zeros((self.B, self.Hkv, self.cap, self.d), np.float32) for _ in range(2))
        Q = np.zeros((self.B, self.Hq, self.d), np.float32)
        th = self.table.cpu().numpy()
        if self.quant:
            kd, vd = (ref.values(t.cpu().numpy(), self.d) for t in (self.kp, self.vp))
        else:
            kd, vd = (t.float().cpu().numpy() for t in (self.kp, self.vp))
        worst = 0.0
        for b, n in enumerate(self.lens):
            pos = np.arange(n)
            kr, _ = ref.rotate(host[b, :n, self.Hq:self.Hq + self.Hkv], tab, pos, False)
            for p in range(n):
                K[b, :, p], V[b, :, p] = kd[th[b, p // C], :, p % C], vd[th[b, p // C], :, p % C]
            g = kr.reshape(n, self.Hkv, -1, 32)
            half = (g.max(-1) - g.min(-1))[..., None] / 30 if self.quant else 2.0 ** -8 * np.abs(g)
            worst = max(worst, np.max((np.abs(K[b, :, :n].transpose(1, 0, 2).reshape(g.shape) - g)) / (half * 1.02 + 1e-2 * self.quant + 1e-6)))
            q, _ = ref.rotate(host[b, n - 1:n, : self.Hq], tab, pos[-1:], False)
            Q[b] = torch.from_numpy(q[0]).bfloat16().float().numpy()
        assert worst <= 1.0, worst                  # the cache holds the rotated keys
        oracle = Oracle(self.B, self.Hq, self.Hkv, self.cap, self.d, C, self.K)
        kp, bp = oracle.summary(K, self.lq.float().cpu().numpy())
        return oracle.decode(Q, K, V, kp, bp, np.array(self.lens)), K, V, kp, bp

    def check(self):
        r, K, V, kp, bp = self.reference()
        ok = r["gap"].reshape(-1) >= SEL_GAP["bf16"]
        err = np.abs(self.o.float().cpu().numpy() - r["O"]).reshape(-1, self.d)[ok]
        assert ok.any() and err.max() <= OUT_MAX["bf16"], err.max()


@pytest.mark.parametrize("quant", [False, True])
def test_serving_loop(quant):
    """Prompts of unequal length (one inside its first chunk, one that ends on a border), then steps over which every
    sequence completes a chunk; each step against the oracle on what the cache holds."""
    loop = _Loop(quant)
    loop.prompt([61, 128, 250])
    for i in range(7):
        loop.feed()
        loop.step()
        assert hils.hils_get_status() == 0
        if i in (0, 2, 3, 6):
            loop.check()


@pytest.mark.parametrize("quant", [False, True])
def test_serving_step_captured_and_replayed(quant):
    """One step captured once and replayed: the outputs of the eager loop, bit for bit, while the eager loop of another
    batch runs between the replays."""
    eager, graphed, other = _Loop(quant), _Loop(quant), _Loop(quant, seed=33)
    for loop, lens in ((eager, [61, 128, 250]), (graphed, [61, 128, 250]), (other, [5, 63, 190])):
        loop.prompt(lens)
    graphed.feed()
    keep = [t.clone() for t in (graphed.kp, graphed.vp, graphed.seqlens)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step()
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip((graphed.kp, graphed.vp, graphed.seqlens), keep):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for i in range(5):
        if i:
            graphed.feed()
        graph.replay()
        other.feed()
        other.step()
        eager.feed()
        eager.step()
        assert torch.equal(graphed.o, eager.o)
    assert torch.equal(graphed.kp, eager.kp) and torch.equal(graphed.vp, eager.vp)
    assert torch.equal(graphed.summ.kprime, eager.summ.kprime)
    assert hils.hils_get_status() == 0


def test_two_loops_on_two_streams():
    """Two batches on streams of their own, launched in turn with stream=: the results of each alone."""
    loops, alone = [_Loop(True, seed=40 + i) for i in range(2)], [_Loop(True, seed=40 + i) for i in range(2)]
    lens = [[61, 128, 250], [200, 3, 127]]
    for a, n in zip(alone, lens):
        a.prompt(n)
        for _ in range(4):
            a.feed()
            a.step()
    streams = [torch.cuda.Stream() for _ in loops]
    for loop, n, st in zip(loops, lens, streams):
        loop.prompt(n, stream=st)
    torch.cuda.synchronize()
    for _ in range(4):
        for loop, st in zip(loops, streams):
            with torch.cuda.stream(st):
                loop.feed()
                loop.seqlens.add_(0)
            loop.seqlens.record_stream(st)
            with torch.cuda.stream(st):
                loop.step()
    for st in streams:
        st.synchronize()
    assert hils.hils_get_status() == 0
    for a, b in zip(loops, alone):
        assert torch.equal(a.o, b.o) and torch.equal(a.kp, b.kp) and torch.equal(a.summ.kprime, b.summ.kprime)


def test_empty_calls_and_default_stream_handles():
    """No tokens: nothing is launched, nothing changes; stream=0 is the default stream."""
    for quant in (False, True):
        loop = _Loop(quant)
        before = hils.hils_kernel_launches()
        none = loop.x[0, :0]
        q, k, v = loop._split(none)
        cu = torch.zeros(loop.B + 1, dtype=torch.int32, device="cuda")
        out = hils.kv_append(loop.kp, loop.vp, loop.table, k, v, loop.seqlens, cu_tokens=cu, rotary=loop.rotary, q=q)
        assert out.shape == (0, loop.Hq, loop.d)
        hils.landmark_summary_append(loop.kp, loop.table, loop.lq, loop.seqlens, 0, loop.summ, cu_tokens=cu)
        if quant:
            k, v = hils.kv_read(loop.kp, loop.vp, loop.table, loop.seqlens, 0, torch.bfloat16)
            assert k.shape == v.shape == (0, loop.Hkv, loop.d)
        assert hils.hils_kernel_launches() == before and bool((loop.kp == 0).all())
    a, b = _Loop(True, seed=60), _Loop(True, seed=60)
    for loop, stream in ((a, None), (b, 0)):
        loop.prompt([61, 128, 250], stream=stream)
        loop.feed()
        loop.step(stream=stream)
    assert torch.equal(a.o, b.o) and hils.hils_get_status() == 0


def test_sequences_that_share_a_prefix():
    """Two sequences whose tables name the same pages for their first chunks, with tails of their own: each decodes as
    if it had the pages alone, and a step's append writes its own tail."""
    loop = _Loop(True, B=2, seed=70)
    loop.x[1, :128] = loop.x[0, :128]
    loop.lq[1, :, :2] = loop.lq[0, :, :2]
    alone = _Loop(True, B=2, seed=70)
    alone.x.copy_(loop.x), alone.lq.copy_(loop.lq)
    alone.prompt([140, 150])
    # the shared form: the second sequence appends only what follows the prefix
    loop.table[1, :2] = loop.table[0, :2]
    rows = torch.cat([loop.x[0, :140], loop.x[1, 128:150]])
    q, k, v = loop._split(rows)
    loop.seqlens.copy_(torch.tensor([140, 150], dtype=torch.int32))
    cu = torch.tensor([0, 140, 162], dtype=torch.int32, device="cuda")
    hils.kv_append(loop.kp, loop.vp, loop.table, k, v, loop.seqlens, cu_tokens=cu, rotary=loop.rotary, q=q)
    hils.landmark_summary_append(loop.kp, loop.table, loop.lq, loop.seqlens, 162, loop.summ, cu_tokens=cu)
    for t in (loop.summ.kprime, loop.summ.bprime, loop.summ.kprime_mma.view(2, loop.Hkv, -1, loop.d + 16)):
        t[1, :, :2] = t[0, :, :2]
    loop.lens = [140, 150]
    for _ in range(3):
        for x in (loop, alone):
            x.feed()
            x.step()
        assert torch.equal(loop.o, alone.o)
    assert hils.hils_get_status() == 0


def test_step_is_reproducible():
    m = _cache(4, 16, 4, 128, 4096, "bf16", seed=50)
    seq = torch.tensor([4096, 4000, 100, 2049], dtype=torch.int32, device="cuda")
    first = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 16, window=128, with_selection=True)
    for _ in range(5):
        again = hils.decode_step_quant(m["q"], m["kp"], m["vp"], m["table"], m["summ"], seq, 16, window=128, with_selection=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
