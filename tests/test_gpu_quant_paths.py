"""Kernels of the 4-bit calls that only certain sizes reach: the top-K that reads its scores again (beyond 32768
candidates) with distinct scores, the summaries of many chunks (a warp per chunk) at both head sizes, and the scores
that a decode step returns."""
import numpy as np
import pytest
import torch

from chunk_wise_sparse_b200 import hils
from oracle.oracle import Oracle, Rows
from tests import paged_reference as ref
from tests.helpers import SUMMARY_TOL

pytestmark = pytest.mark.gpu

C = 64


@pytest.mark.parametrize("nc,K", [(33000, 16), (33001, 64), (40003, 1), (9000, 16), (32768, 64), (8192, 3), (2048, 5),
                                  (2049, 64)])
def test_distinct_scores_of_long_rows(nc, K):
    """Scores are the entropy biases (the queries are zero): any order of distinct numbers, the K largest of which are
    kept with their ids ascending, for rows of every kernel variant."""
    rng = np.random.default_rng(nc)
    cap = nc * C
    kp, vp = hils.quant_pages(1, 1, 64), hils.quant_pages(1, 1, 64)
    table = torch.zeros((1, nc), dtype=torch.int32, device="cuda")      # every chunk is the one page
    bias = rng.permutation(nc).astype(np.float32) / 8 - 100             # exact in fp32
    summ = hils.Summary.of(torch.zeros((1, 1, nc, 64), device="cuda"), torch.from_numpy(bias).cuda().view(1, 1, nc))
    q = torch.zeros((1, 2, 64), device="cuda")
    for n in (cap, cap - 64 * (nc // 3) - 5, 64 * (K + 1) + 1):
        seq = torch.tensor([n], dtype=torch.int32, device="cuda")
        _, ids, sc = hils.decode_step_quant(q, kp, vp, table, summ, seq, K, with_selection=True)
        assert hils.hils_get_status() == 0
        cand = bias[:(n - 1) // C]
        want = np.sort(np.argsort(-cand, kind="stable")[:K])
        for row in range(2):
            assert np.array_equal(ids[0, row].cpu().numpy(), want)
            assert np.array_equal(sc[0, row].cpu().numpy(), cand[want])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,H,chunks", [(64, 1, 700), (128, 1, 700), (64, 5, 600), (128, 5, 600), (64, 8, 1900),
                                        (128, 8, 1900), (64, 3, 8000), (128, 4, 8000)])
def test_summaries_of_prompts(dtype, d, H, chunks):
    """Prompts of so many chunks that a warp has one each, one to four chunks per CTA, the last CTA's heads and chunks
    not all there, two sequences that meet inside a CTA's tokens."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(d + H)
    a = chunks * 2 // 3
    lens = [a * C + 17, (chunks - a) * C]
    nc, n_pages = max(-(-n // C) for n in lens), 97
    pages = ref.pack(rng.standard_normal((n_pages, H, C, d)).astype(np.float32))
    dense = torch.from_numpy(ref.values(pages, d)).cuda().double()
    table = torch.from_numpy(rng.integers(0, n_pages, (2, nc)).astype(np.int32)).cuda()      # pages are read only: shared
    lq = torch.from_numpy(rng.standard_normal((2, H, nc, d)).astype(np.float32)).to(dt).cuda()
    summ = hils.Summary(hils.make_dims(2, H, H, d, nc * C, 1, dt), "cuda")
    for t in (summ.kprime, summ.bprime, summ.kprime_mma):
        if t is not None:
            t.fill_(11.0)
    hils.landmark_summary_append(torch.from_numpy(pages).cuda(), table, lq,
                                 torch.tensor(lens, dtype=torch.int32, device="cuda"), sum(lens), summ,
                                 cu_tokens=torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda"))
    assert hils.hils_get_status() == 0
    for b, n in enumerate(lens):
        done = n // C
        for h in range(H):
            k = dense[table[b, :done].long(), h]                                   # [chunks, 64, d]
            p = (torch.einsum("cjd,cd->cj", k, lq[b, h, :done].double()) / d ** 0.5).softmax(-1)
            kp, bp = torch.einsum("cj,cjd->cd", p, k), -(p * p.log()).sum(-1)
            assert (summ.kprime[b, h, :done] - kp).abs().max().item() <= SUMMARY_TOL
            assert (summ.bprime[b, h, :done] - bp).abs().max().item() <= SUMMARY_TOL
        assert bool((summ.kprime[b, :, done:] == 11.0).all()) and bool((summ.bprime[b, :, done:] == 11.0).all())
        if summ.kprime_mma is not None:
            m = summ.kprime_mma.view(2, H, nc, d + 16)[b]
            assert torch.equal(m[:, :done, :d], summ.kprime[b, :, :done].bfloat16())
            got = m[:, :done, d].double() + m[:, :done, d + 1].double()
            want = summ.bprime[b, :, :done].double() * d ** 0.5
            # two bf16 values: the second is rounded to 2^-8 of itself, itself at most 2^-8 of the sum
            assert bool(((got - want).abs() <= 2.0 ** -16 * want.abs() + 1e-5).all())
            assert bool((m[:, :done, d + 2:] == 0).all()) and bool((m[:, done:] == 11.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,Hq,Hkv,window", [(64, 8, 2, 0), (128, 6, 2, 192), (128, 16, 1, 0)])
def test_returned_scores(dtype, d, Hq, Hkv, window):
    """The scores of the kept chunks, against the oracle's of the same chunks.

    fp32: sums of d + 1 products in fp32, each at most (d + 1) 2^-24 of tau sum |q||k'| + |b'|.  bf16: the operand
    rounds k' by 2^-8 of each value (b' / tau is a sum of two, within 2^-16 of it)."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, cap, K = 2, 2048, 8
    nc, rng = cap // C, np.random.default_rng(d + Hq)
    pools, dense = [], []
    table = rng.permutation(B * nc + 2)[: B * nc].astype(np.int32).reshape(B, nc)
    for _ in range(2):
        p = ref.pack(rng.standard_normal((B * nc + 2, Hkv, C, d)).astype(np.float32))
        dense.append(np.ascontiguousarray(ref.values(p, d)[table.reshape(-1)].reshape(B, nc, Hkv, C, d)
                                          .transpose(0, 2, 1, 3, 4).reshape(B, Hkv, cap, d)))
        pools.append(torch.from_numpy(p).cuda())
    q = torch.from_numpy(rng.standard_normal((B, Hq, d)).astype(np.float32)).to(dt).cuda()
    lq = torch.from_numpy(rng.standard_normal((B, Hkv, nc, d)).astype(np.float32)).to(dt).cuda()
    tab = torch.from_numpy(table).cuda()
    summ = hils.Summary(hils.make_dims(B, Hkv, Hkv, d, cap, 1, dt), "cuda")
    hils.landmark_summary_append(pools[0], tab, lq, torch.full((B,), cap, dtype=torch.int32, device="cuda"), B * cap, summ)
    lens = np.array([cap, 1500])
    _, ids, sc = hils.decode_step_quant(q, pools[0], pools[1], tab, summ, torch.from_numpy(lens.astype(np.int32)).cuda(),
                                        K, window=window, with_selection=True)
    assert hils.hils_get_status() == 0
    oracle = Oracle(B, Hq, Hkv, cap, d, C, K, window)
    kp, bp = oracle.summary(dense[0], lq.float().cpu().numpy())
    qh = q.float().cpu().numpy()
    want = np.take_along_axis(oracle.scores(kp, bp, Rows.from_decode(qh, lens)), ids.view(-1, K).cpu().numpy(), -1)
    G, tau = Hq // Hkv, 1 / np.sqrt(d)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for r, (b, hq) in enumerate(np.ndindex(B, Hq)):
        c = ids[b, hq].cpu().numpy()
        mag = tau * (np.abs(kp[b, hq // G, c]) @ np.abs(qh[b, hq])) + np.abs(bp[b, hq // G, c])
        tol = half * tau * (np.abs(kp[b, hq // G, c]) @ np.abs(qh[b, hq])) + (2.0 ** -16 if dtype == "bf16" else 0) * np.abs(bp[b, hq // G, c])
        # the summaries' own tolerance enters each product
        tol = tol + (d + 1) * 2.0 ** -24 * mag + SUMMARY_TOL * (1 + tau * np.abs(qh[b, hq]).sum())
        assert np.all(np.abs(sc[b, hq].cpu().numpy() - want[r]) <= tol)
