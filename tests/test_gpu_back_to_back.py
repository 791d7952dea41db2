"""Decode steps launched back to back on one workspace, so that what a step's kernels read was last written by another
step: each output is the one of the step alone, on a workspace that held garbage before."""
import pytest
import torch

from chunk_wise_sparse_b200 import hils

pytestmark = pytest.mark.gpu

C, STEPS = 64, 12


@pytest.mark.parametrize("kind", ["bf16", "fp32", "bf16-4bit", "fp32-4bit"])
@pytest.mark.parametrize("B,Hq,Hkv,d,nc,K,window", [
    (3, 8, 2, 64, 40, 8, 0),             # rows in registers
    (2, 4, 2, 128, 4500, 16, 128),       # longer rows
    (1, 4, 1, 64, 9000, 32, 0),          # rows that an unquantised step reads from memory again
    (1, 2, 1, 64, 33000, 3, 512),        # and a 4-bit step
    (2, 4, 4, 64, 8, 16, 64),            # fewer candidates than are kept
])
def test_steps_share_a_workspace(kind, B, Hq, Hkv, d, nc, K, window):
    dt = torch.bfloat16 if kind.startswith("bf16") else torch.float32
    quant = kind.endswith("4bit")
    g = torch.Generator("cuda").manual_seed(nc)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731
    cap, n_pages = nc * C, 64
    table = torch.randint(0, n_pages, (B, nc), device="cuda", generator=g).to(torch.int32)     # pages are read only
    if quant:
        kp, vp = hils.quant_pages(n_pages, Hkv, d), hils.quant_pages(n_pages, Hkv, d)
        every = torch.arange(n_pages, dtype=torch.int32, device="cuda").view(1, -1)
        hils.kv_append(kp, vp, every, normal(n_pages * C, Hkv, d).to(dt), normal(n_pages * C, Hkv, d).to(dt),
                       torch.tensor([n_pages * C], dtype=torch.int32, device="cuda"))
    else:
        kp, vp = normal(n_pages, Hkv, C, d).to(dt), normal(n_pages, Hkv, C, d).to(dt)
    dims = hils.make_dims(B, Hq, Hkv, d, cap, K, dt, window=window)
    summ = hils.Summary(dims, "cuda")
    summ.kprime.copy_(normal(B, Hkv, nc, d)), summ.bprime.copy_(normal(B, Hkv, nc))
    if dt == torch.bfloat16:
        m = summ.kprime_mma.view(B, Hkv, nc, d + 16)
        m.copy_(normal(B, Hkv, nc, d + 16))
        m[..., d + 2:] = 0
    qs = [normal(B, Hq, d).to(dt) for _ in range(STEPS)]
    lens = [torch.randint(max(1, cap - 700), cap + 1, (B,), device="cuda", generator=g).to(torch.int32) for _ in range(STEPS)]
    need = hils.hils_decode_quant_workspace_bytes if quant else hils.hils_decode_workspace_bytes
    ws = torch.empty((need(dims),), dtype=torch.uint8, device="cuda")

    def new():
        return [(torch.empty_like(q), torch.empty((B, Hq, K), dtype=torch.int32, device="cuda"),
                 torch.empty((B, Hq, K), device="cuda")) for q in qs]

    call = hils.hils_attn_decode_quant if quant else None

    def step(i, out):
        o, ids, sc = out[i]
        if call:
            call(dims, qs[i], None, kp, vp, table, n_pages, summ.kprime, summ.bprime, summ.kprime_mma, lens[i], o, ids,
                 sc, ws)
        else:
            hils.hils_attn_decode_paged(dims, qs[i], kp, vp, table, n_pages, summ.kprime, summ.bprime, summ.kprime_mma,
                                        lens[i], o, ids, sc, ws)

    want = new()
    for i in range(STEPS):
        ws.fill_(0xFF)                  # NaN scores, ids of -1
        torch.cuda.synchronize()
        step(i, want)
        torch.cuda.synchronize()
    got = new()
    for i in range(STEPS):
        step(i, got)
    replayed = new()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(STEPS):
            step(i, replayed)
    for _ in range(3):
        graph.replay()
    assert hils.hils_get_status() == 0
    for out in (got, replayed):
        for a, b in zip(want, out):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
