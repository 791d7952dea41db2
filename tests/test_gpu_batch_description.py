"""Batch descriptions that do not fit (cu_tokens beyond the packed tokens, or not ascending): recorded, and the tokens of
the sequences concerned are skipped, so that nothing already in the cache changes."""
import pytest
import torch

from chunk_wise_sparse_b200 import hils

pytestmark = pytest.mark.gpu

C = 64
T, B, HQ, HKV, D, CAP = 16, 4, 4, 2, 64, 128
GOOD = [0, 3, 5, 10, 16]
LENS = [10, 66, 128, 70]

# (cu_tokens, the sequences that fit)
BAD = [
    ([0, 3, 5, 10, 17], [0, 1, 2]),      # the last one reaches beyond the packed tokens
    ([0, 3, 5, 18, 18], [0, 1]),         # one in the middle does, and an empty one behind it
    ([0, 3, 2, 10, 16], [3]),            # a descent: sequences 0 .. 2 touch it
    ([0, 3, 12, 10, 16], [0]),           # sequences 1 .. 3 touch it
    ([1, 3, 5, 10, 16], [1, 2, 3]),      # does not start at 0: sequence 0 would lack a token
    ([-2, 3, 5, 10, 16], [1, 2, 3]),
    ([0, 3, 5, 10, 4], [0]),             # the tokens end inside sequence 1
]


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class _State:
    def __init__(self, quant):
        g = torch.Generator("cuda").manual_seed(4)
        n = B * CAP // C + 2
        self.quant = quant
        self.table = torch.randperm(n, device="cuda", generator=g)[: B * CAP // C].to(torch.int32).view(B, -1)
        self.q, self.k, self.v = (torch.randn((T, h, D), device="cuda", generator=g).bfloat16() for h in (HQ, HKV, HKV))
        self.rotary = hils.Rotary(hils.rotary_table(CAP, D))
        shape, kind = ((n, HKV, C * 40), torch.uint8) if quant else ((n, HKV, C, D), torch.bfloat16)
        self.shape, self.kind = shape, kind
        self.lq = torch.randn((B, HKV, CAP // C, D), device="cuda", generator=g).bfloat16()
        if quant:       # rows to summarise and to read back
            self.kp, self.vp = hils.quant_pages(n, HKV, D), hils.quant_pages(n, HKV, D)
            x = torch.randn((B * CAP, HKV, D), device="cuda", generator=g).bfloat16()
            hils.kv_append(self.kp, self.vp, self.table, x, x, _int([CAP] * B))

    def append(self, cu):
        kp, vp = (torch.full(self.shape, 9, dtype=self.kind, device="cuda") for _ in range(2))
        q = torch.full_like(self.q, 3.0)
        hils.kv_append(kp, vp, self.table, self.k, self.v, _int(LENS), cu_tokens=_int(cu), rotary=self.rotary, q=self.q,
                       q_out=q)
        return kp, vp, q

    def read(self, cu):
        k, v = torch.full_like(self.k, 3.0), torch.full_like(self.k, 3.0)
        hils.kv_read(self.kp, self.vp, self.table, _int(LENS), T, torch.bfloat16, cu_tokens=_int(cu), k_out=k, v_out=v)
        return k, v

    def summary(self, cu):
        summ = hils.Summary(hils.make_dims(B, HKV, HKV, D, CAP, 1, torch.bfloat16), "cuda")
        for t in (summ.kprime, summ.bprime, summ.kprime_mma):
            t.fill_(11.0)
        hils.landmark_summary_append(self.kp, self.table, self.lq, _int(LENS), T, summ, cu_tokens=_int(cu))
        return summ.kprime, summ.bprime


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("cu,fit", BAD)
def test_append_skips_the_sequences_that_do_not_fit(quant, cu, fit):
    s = _State(quant)
    kp, vp, q = s.append(GOOD)
    assert hils.hils_get_status() == 0
    kp2, vp2, q2 = s.append(cu)
    assert hils.hils_get_status() == 6
    keep = torch.zeros(T, dtype=torch.bool, device="cuda")
    for b in fit:
        keep[GOOD[b]:GOOD[b + 1]] = True
    assert torch.equal(q2[keep], q[keep]) and bool((q2[~keep] == 3.0).all())
    for got, want in ((kp2, kp), (vp2, vp)):
        for b in range(B):
            pages = s.table[b].long()
            assert torch.equal(got[pages], want[pages]) if b in fit else bool((got[pages] == 9).all()), b


@pytest.mark.parametrize("cu,fit", BAD)
def test_read_back_and_summaries_skip_them_too(cu, fit):
    s = _State(True)
    k, v = s.read(GOOD)
    kprime, bprime = s.summary(GOOD)
    assert hils.hils_get_status() == 0
    assert bool((kprime[2, :, 1] != 11.0).all())         # sequence 2 completes its second chunk
    k2, v2 = s.read(cu)
    assert hils.hils_get_status() == 6
    kprime2, bprime2 = s.summary(cu)
    assert hils.hils_get_status() == 6
    for b in range(B):
        at = slice(GOOD[b], GOOD[b + 1])
        if b in fit:
            assert torch.equal(k2[at], k[at]) and torch.equal(v2[at], v[at])
            assert torch.equal(kprime2[b], kprime[b]) and torch.equal(bprime2[b], bprime[b])
        else:
            assert bool((k2[at] == 3.0).all()) and bool((v2[at] == 3.0).all())
            assert bool((kprime2[b] == 11.0).all()) and bool((bprime2[b] == 11.0).all())
