"""The bf16 decode step over 4-bit pages at value scales from 1e-4 to 1e4, against a 64-bit definition on what the pages
and the scoring operand stand for.

Tolerances.  An output is o_i = sum_j w_j (m_j + s_j code_ji), sum_j w_j = 1.  The kernel rounds a weight to fp16 (half a
step: 2^-11 of it) and its product with the step once more (another 2^-11), the result to bf16 (2^-8 of it); the sums
are fp32.  So a key's term is off by at most
    h_ji = w_j (2^-10 s_j code_ji + 2^-11 |m_j|) (1 + 2^-8)
and, where the weight or its product falls below fp16's normal range, by half of fp16's least step: with weights scaled
by 2^k that is 2^-25 2^-k (15 for a product with a code of at most 15, 15 s_j + |m_j| for a weight), for each of n keys.
The weights (at most 1) are scaled as far as their products with the largest step stay below 2^15, by 2^15 at most:
k = min(15, 14 - floor(log2 max s)).
A logit is a sum of at most 2 (d / 16 + 1) products of 16 terms whose addends the matrix unit cuts to 24 bits or more,
and d / 16 fp32 steps: off by at most 17 (d / 8 + 2 + d / 16) 2^-24 A <= 17 (3 d / 16 + 2) 2^-24 A with
A = tau sum_i |q_i| (s code_i + |m|); a weight by twice that.  Rounding errors of different keys are independent, so over
many outputs their root mean square is at most that of sqrt(sum_j h_ji^2).
"""
import math

import numpy as np
import pytest
import torch

from chunk_wise_sparse_b200 import hils
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu

C = 64


def _decode(d, cap, K, window, lens, k_rows, v_rows, q, seed):
    """One step over 4-bit pages of the rows k_rows, v_rows [n_pages, Hkv, 64, d]; everything the definition needs."""
    rng = np.random.default_rng(seed)
    B, Hq, _ = q.shape
    n_pages, Hkv = k_rows.shape[:2]
    nc = cap // C
    table = rng.permutation(n_pages)[: B * nc].astype(np.int32).reshape(B, nc)
    kp, vp = (torch.from_numpy(ref.pack(x)).cuda() for x in (k_rows, v_rows))
    qt = torch.from_numpy(q.astype(np.float32)).bfloat16().cuda()
    lq = torch.from_numpy(rng.standard_normal((B, Hkv, nc, d)).astype(np.float32)).bfloat16().cuda()
    tab = torch.from_numpy(table).cuda()
    summ = hils.Summary(hils.make_dims(B, Hkv, Hkv, d, cap, 1, torch.bfloat16), "cuda")
    full = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    hils.landmark_summary_append(kp, tab, lq, full, B * cap, summ)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, ids, _ = hils.decode_step_quant(qt, kp, vp, tab, summ, seq, K, window=window, with_selection=True)
    assert hils.hils_get_status() == 0
    return (o.double().cpu().numpy(), ids.cpu().numpy(), qt.double().cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy(),
            table, summ.kprime_mma.view(B, Hkv, nc, d + 16).double().cpu().numpy())


def _definition(ids, q, kp, vp, table, mma, d, K, window, lens):
    """(o, root of the summed squares of h, sum of h, error of the logits' part) of the step, in 64 bits."""
    B, Hq, _ = q.shape
    Hkv = kp.shape[1]
    G, wc, root = Hq // Hkv, max(1, window // C), math.sqrt(d)
    kc, ks, km = ref.unpack(kp, d)
    vc, vs, vm = ref.unpack(vp, d)
    wide = lambda x: np.repeat(x, ref.GROUP, -1)  # noqa: E731
    k = min(15, 14 - math.floor(math.log2(vs.max())))
    under = 2.0 ** (-25 - k) * (15 + 15 * vs.max() + np.abs(vm).max())
    o, rms, top, logit = (np.zeros((B, Hq, d)) for _ in range(4))
    for b, n in enumerate(lens):
        own = (n - 1) // C
        for hq in range(Hq):
            h, x = hq // G, q[b, hq]
            w, v, s_code, least, A = [], [], [], [], 0.0
            branches = [(int(c), None) for c in ids[b, hq] if c >= 0]
            near = [c for c in range(max(0, own - wc + 1), own + 1)]
            for c, _ in branches + [(c, "window") for c in near]:
                page = table[b, c]
                m = min(C, n - c * C)
                key = (wide(km[page, h]) + wide(ks[page, h]) * kc[page, h])[:m]
                A = max(A, float(((wide(np.abs(km[page, h])) + wide(ks[page, h]) * kc[page, h])[:m] @ np.abs(x)).max()) / root)
                e = np.exp(key @ x / root)
                if c in near:
                    w.append(e)                     # the window is one branch: its weight is the sum of its exponentials
                else:
                    r = mma[b, h, c]
                    w.append(math.exp((r[:d] @ x + r[d] + r[d + 1]) / root) * e / e.sum())
                v.append((wide(vm[page, h]) + wide(vs[page, h]) * vc[page, h])[:m])
                s_code.append((wide(vs[page, h]) * vc[page, h])[:m])
                least.append(wide(np.abs(vm[page, h]))[:m])
            w, v, s_code, least = np.concatenate(w), np.concatenate(v), np.concatenate(s_code), np.concatenate(least)
            w = w / w.sum()
            o[b, hq] = w @ v
            term = w[:, None] * (2.0 ** -10 * s_code + 2.0 ** -11 * least) * (1 + 2.0 ** -8)
            rms[b, hq], top[b, hq] = np.sqrt((term ** 2).sum(0)), term.sum(0) + len(w) * under
            logit[b, hq] = 2 * 17 * (3 * d / 16 + 2) * 2.0 ** -24 * A * (w @ np.abs(v))
    return o, rms, top, logit


SCALES = [1.0, 1e-2, 1e-3, 1e-4]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", SCALES)
def test_equal_rows_are_returned_at_every_scale(d, scale):
    """All rows of values are one ramp and all weights are equal, so that the roundings of all keys add up: the output
    is the ramp."""
    cap, n_pages, K = 1024, 17, 8
    rng = np.random.default_rng(d)
    k = rng.standard_normal((n_pages, 1, C, d)).astype(np.float32)
    row = np.resize(np.linspace(-1, 1, 32), d) * scale
    v = np.broadcast_to(row, k.shape).astype(np.float32)
    q = np.zeros((1, 4, d))
    got = _decode(d, cap, K, 0, [cap], k, v, q, seed=d)
    o, _, top, logit = _definition(*got[1:], d, K, 0, [cap])
    assert np.abs(o - row).max() <= 0.075 * scale      # half a step of 2 / 15, and its rounding to fp16 at 1e-4
    assert np.all(np.abs(got[0] - o) <= 2.0 ** -8 * np.abs(o) + top + logit)


@pytest.mark.parametrize("d,Hq,Hkv,K,window,lens", [
    (64, 8, 2, 16, 0, [4096, 4051]), (128, 8, 2, 16, 512, [4096, 3969]), (128, 2, 2, 64, 0, [8192, 6000]),
])
@pytest.mark.parametrize("scale", SCALES + [1e4])
def test_random_values_at_every_scale(d, Hq, Hkv, K, window, lens, scale):
    """Values of one spread: every output within the sum of the bounds, and the root mean square within theirs."""
    B, cap = len(lens), -(-max(lens) // C) * C
    rng = np.random.default_rng(d + K)
    n_pages = B * (cap // C) + 3
    k = rng.standard_normal((n_pages, Hkv, C, d)).astype(np.float32)
    v = (rng.standard_normal((n_pages, Hkv, C, d)) * scale).astype(np.float32)
    got = _decode(d, cap, K, window, lens, k, v, rng.standard_normal((B, Hq, d)), seed=d)
    o, rms, top, logit = _definition(*got[1:], d, K, window, lens)
    err = np.abs(got[0] - o)
    assert np.all(err <= 2.0 ** -8 * np.abs(o) + top + logit)
    want = np.sqrt((rms ** 2).mean()) + 2.0 ** -8 * np.sqrt((o ** 2).mean()) + np.sqrt((logit ** 2).mean())
    assert np.sqrt((err ** 2).mean()) <= want


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_unlike_chunks(d):
    """Neighbouring chunks whose values differ by 2^20 in scale, large and small ones in any order, groups of zero steps
    between them."""
    cap, n_pages, K = 2048, 35, 24
    rng = np.random.default_rng(7 * d)
    scale = np.exp2(rng.integers(-14, 7, n_pages)).astype(np.float32)[:, None, None, None]
    k = rng.standard_normal((n_pages, 2, C, d)).astype(np.float32)
    v = rng.standard_normal((n_pages, 2, C, d)).astype(np.float32) * scale
    v[::3, :, :, :32] = v[::3, :, :1, :1]
    got = _decode(d, cap, K, 128, [cap, cap - 70], np.concatenate([k, k]), np.concatenate([v, v]),
                  rng.standard_normal((2, 6, d)), seed=d)
    o, _, top, logit = _definition(*got[1:], d, K, 128, [cap, cap - 70])
    assert np.all(np.abs(got[0] - o) <= 2.0 ** -8 * np.abs(o) + top + logit)
