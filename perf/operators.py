"""The operators of serving from a chunk-paged cache, as they are measured.

Five operators, the steps of one serving loop:

  append    new keys and values rotated and written into bf16 / fp32 chunk pages, new queries rotated beside them
  append4   the same into pages that hold 4 bits per value; the rows that were written are read back, since what a
            4-bit cache holds is compared as the values it stands for
  read4     rows of a 4-bit cache read back as dense keys and values (a cached prefix handed to the prefill)
  summary   the landmark summaries (k', b', scoring operand) of the chunks that an append completed
  decode4   one decode step of the hierarchical sparse attention over a 4-bit cache

Every operator takes the ragged batch in the same form: `seqlens` [B], the lengths after the append, and the packed new
tokens [T], of sequence b the tokens cu_tokens[b] .. cu_tokens[b + 1] - 1.

A 4-bit page holds, for each kv head, 64 rows of codes and then 64 rows of (step, least value) pairs in fp16, one pair
for 32 dims.  A row of codes is d / 2 bytes: its 16-bit unit e * (d / 32) + g holds the dims 32 g + 4 e .. + 3, the
lowest in the lowest bits.  A code c stands for least + step * c.

Sizes: 16 or 32 query heads, 8 or 16 kv heads, head dims 64 and 128, top-K 16 and 32, 32K / 128K / 512K tokens and
the window of 512 are this repository's own workloads; batches of 64 single tokens are a serving step.
"""
import math
import random

import torch

own = False

CHUNK, GROUP, EXT = 64, 32, 16
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the smallest call: one new token of one sequence, an fp32 model
        _case("append-1-fp32-d64", "append", dtype="fp32", B=1, Hq=16, Hkv=16, d=64, cap=1024, new=1, rot=64,
              interleaved=True),
        # a decode step of 64 sequences, q, k, v being views of one fused projection
        _case("append-step-b64-gqa4-d128", "append", B=64, Hq=32, Hkv=8, d=128, cap=1024, new=1, ragged=3, rot=128,
              fused=True),
        # a whole prompt of the 32K workload, half of the dims rotated (the rest carries no position)
        _case("append-prompt-32k-h16-d64", "append", B=1, Hq=16, Hkv=16, d=64, cap=32768, new=32768, rot=32, fused=True),
        # the decode step into a 4-bit cache
        _case("append4-step-b64-gqa4-d128", "append4", B=64, Hq=32, Hkv=8, d=128, cap=4096, new=1, ragged=5, rot=128,
              fused=True),
        # pieces of eight prompts of unequal length
        _case("append4-ragged-b8-gqa4-d128", "append4", B=8, Hq=32, Hkv=8, d=128, cap=16384, new=2047, ragged=7, rot=64,
              interleaved=True),
        # a short cached prefix of three sequences
        _case("read4-ragged-b3-d64", "read4", B=3, Hq=4, Hkv=4, d=64, cap=2048, new=301, ragged=11),
        # the whole prefix of a 128K sequence
        _case("read4-128k-gqa4-d128", "read4", B=1, Hq=32, Hkv=8, d=128, cap=131072, new=131072),
        # a decode step in which a few of 64 sequences complete a chunk
        _case("summary-step-b64-d128", "summary", B=64, Hq=32, Hkv=8, d=128, cap=1024, new=1, ragged=15),
        # a whole prompt in 4 bits
        _case("summary4-prompt-128k-h16-d64", "summary", quant=True, B=1, Hq=16, Hkv=16, d=64, cap=131072, new=131072),
        # the smallest decode: three short sequences of unequal length, an fp32 model, a local window
        _case("decode4-b3-h8-d64-fp32-w256", "decode4", dtype="fp32", B=3, Hq=8, Hkv=4, d=64, cap=4096, ragged=17, K=8,
              window=256),
        # the batch decode workload: 8 sequences of 128K, 4 query heads per kv head
        _case("decode4-128k-b8-gqa4-d128", "decode4", B=8, Hq=32, Hkv=8, d=128, cap=131072, K=32),
        # the 512K workload's decode step
        _case("decode4-512k-h16-d64", "decode4", B=1, Hq=16, Hkv=16, d=64, cap=524288, K=16),
    ]


def _case(name, op, *, dtype="bf16", quant=False, B, Hq, Hkv, d, cap, new=0, ragged=0, rot=0, interleaved=False,
          fused=False, K=16, window=0):
    c = dict(op=op, dtype=dtype, quant=quant or op in ("append4", "read4", "decode4"), B=B, Hq=Hq, Hkv=Hkv, d=d, cap=cap,
             new=new, ragged=ragged, rot=rot, interleaved=interleaved, fused=fused, K=K, window=window)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "append4", "read4", "summary", "decode4", "decode4"])
    d, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8])
    # fp32: a 4-bit cache read back in fp32 shows a code that lies on the border of two as a whole step, so the fp32
    # draws are of the exact append and of the decode, whose selection is far from borders at these lengths
    dtype = rng.choice(["bf16", "bf16", "fp32"]) if op == "append" else "bf16"
    ragged = rng.randrange(1, 1 << 20)
    if op == "decode4":
        K, window = rng.choice([1, 4, 8, 16, 24, 32, 64]), rng.choice([0, 0, 64, 192, 512, 1024])
        B = _log_int(rng, 1, 16)
        most = min(524288, (8 * 8 * 131072 * 128) // (B * Hkv * d))
        cap = CHUNK * _log_int(rng, 4, max(4, most // CHUNK))
        return _case(None, op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, cap=cap, ragged=ragged if rng.random() < 0.7 else 0, K=K,
                     window=window)
    B = _log_int(rng, 1, 64)
    heads = Hkv * (G + 2) if op.startswith("append") else 2 * Hkv
    tokens = (32768 * 48 * 64) // (heads * d) if op.startswith("append") else (131072 * 8 * 128) // (Hkv * d) // 2
    new = _log_int(rng, 1, max(1, min(tokens, 131072) // B // 2))
    cap = min(CHUNK * -(-(2 * new + rng.randrange(1, 4 * CHUNK)) // CHUNK), 262144)
    if op == "read4":  # the pool is what the largest case reads at most
        cap = min(cap, max(CHUNK, 262144 * 1024 // (B * Hkv * d) // CHUNK * CHUNK))
    new = min(new, cap)
    quant = op != "append" and (op != "summary" or rng.random() < 0.6)
    rot = rng.choice([0, 16, d // 4, d // 2, 48, d])
    return _case(None, op, dtype=dtype, quant=quant, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, cap=cap, new=new, ragged=ragged,
                 rot=rot if op.startswith("append") else 0, interleaved=rng.random() < 0.5,
                 fused=rng.random() < 0.5)


def _batch(c):
    """(length before, new tokens) of each sequence.  Part of the case: work() counts with them."""
    if c["op"] == "decode4":
        if not c["ragged"]:
            return [(c["cap"] - 1, 1)] * c["B"]
        r = random.Random(c["ragged"])
        return [(r.randrange(c["cap"]), 1) for _ in range(c["B"])]
    if not c["ragged"]:
        return [(c["cap"] - c["new"], c["new"])] * c["B"]
    r = random.Random(c["ragged"])
    got = []
    for _ in range(c["B"]):
        n = min(c["cap"], r.randint(1, 2 * c["new"] - 1))
        got.append((r.randint(0, c["cap"] - n), n))
    if c["op"] == "summary":   # one chunk at least is completed
        n = got[0][1]
        got[0] = (-(-sum(got[0]) // CHUNK) * CHUNK - n, n)
    return got


def _row_bytes(c):
    return c["d"] // 2 + c["d"] // 8 if c["quant"] else c["d"] * TYPES[c["dtype"]].itemsize


def work(c):
    e, d, batch = TYPES[c["dtype"]].itemsize, c["d"], _batch(c)
    T = sum(n for _, n in batch)
    Hq, Hkv = c["Hq"], c["Hkv"]
    if c["op"] in ("append", "append4"):
        moved = T * (Hq + 2 * Hkv) * d * e + T * c["rot"] * 4 + T * Hq * d * e + 2 * T * Hkv * _row_bytes(c)
        flops = 3 * c["rot"] * T * (Hq + Hkv)
        if c["op"] == "append4":  # and the rows read back; min, max, two operations per code, two per value
            moved += 2 * T * Hkv * (_row_bytes(c) + d * e)
            flops += 2 * T * Hkv * d * 6
        return {"bytes": moved, "flops": flops}
    if c["op"] == "read4":
        return {"bytes": 2 * T * Hkv * (_row_bytes(c) + d * e), "flops": 4 * T * Hkv * d}
    if c["op"] == "summary":
        chunks = sum((s + n) // CHUNK - s // CHUNK for s, n in batch) * Hkv
        return {"bytes": chunks * (CHUNK * _row_bytes(c) + d * e + 4 * d + 4 + 2 * (d + EXT)) + 8 * len(batch),
                "flops": chunks * CHUNK * 4 * d}
    # decode4: the scoring rows of every candidate, and the chunks that at least one of the G heads keeps, each once
    # (expected number for heads that choose independently)
    G, wc, moved, flops = Hq // Hkv, max(1, c["window"] // CHUNK), 2 * c["B"] * Hq * d * e, 0
    for s, _ in batch:
        cand = max(0, s // CHUNK - wc + 1)
        kept = min(c["K"], cand)
        distinct = cand * (1 - (1 - kept / cand) ** G) if cand else 0
        distinct += min(wc, s // CHUNK + 1)
        row = 2 * (d + EXT) if c["dtype"] == "bf16" else 4 * (d + 1)
        moved += Hkv * (cand * row + distinct * 2 * CHUNK * _row_bytes(c))
        flops += Hq * (2 * d * cand + 4 * d * CHUNK * (kept + wc))
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------- inputs

def _codes(x):
    """4-bit codes of x [..., d] by groups of 32 dims: (codes, step, least), in x's own precision; step and least are
    rounded to fp16."""
    g = x.unflatten(-1, (-1, GROUP))
    low = g.amin(-1, keepdim=True).half().to(x.dtype)
    step = ((g.amax(-1, keepdim=True) - g.amin(-1, keepdim=True)) / 15).half().to(x.dtype)
    q = torch.where(step > 0, ((g - low) / torch.where(step > 0, step, 1)).round().clamp(0, 15), 0)
    return q, step, low


def _pack_row(x):
    """(code bytes [..., d / 2], pairs as bytes [..., d / 8]) of rows x [..., d]."""
    q, step, low = _codes(x)
    q = q.unflatten(-1, (8, 4)).transpose(-3, -2).to(torch.uint8)             # [..., e, g, 4]
    codes = (q[..., 0::2] | (q[..., 1::2] << 4)).flatten(-3)
    pairs = torch.cat([step, low], -1).half().flatten(-2).view(torch.uint8)
    return codes, pairs


def _unpack_block(block, d, dtype):
    """Rows [..., 64, d] of blocks [..., 64 * (d / 2 + d / 8)] in `dtype`."""
    n = CHUNK * d // 2
    codes = block[..., :n].unflatten(-1, (CHUNK, 8, d // GROUP, 2))
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).transpose(-3, -2)   # [..., 64, g, e, 4]
    pairs = block[..., n:].contiguous().view(torch.float16).unflatten(-1, (CHUNK, d // GROUP, 2)).to(dtype)
    return (pairs[..., 1:] + pairs[..., :1] * q.flatten(-2).to(dtype)).flatten(-2)


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt, B, Hq, Hkv, d = TYPES[c["dtype"]], c["B"], c["Hq"], c["Hkv"], c["d"]
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    batch = _batch(c)
    T, nc = sum(n for _, n in batch), c["cap"] // CHUNK
    n_pages = B * nc + 5
    s = {"case": c, "T": T, "n_pages": n_pages, "dtype": dt}
    s["seqlens"] = torch.tensor([a + n for a, n in batch], dtype=torch.int32, device="cuda")
    starts = [0]
    for _, n in batch:
        starts.append(starts[-1] + n)
    s["cu"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    # every chunk of every sequence has a page of its own, in no order
    s["table"] = torch.randperm(n_pages, device="cuda", generator=gen)[: B * nc].to(torch.int32).view(B, nc)
    if c["op"].startswith("append"):
        # keys have channels of their own mean, as a model's do
        x = normal(T, Hq + 2 * Hkv, d)
        x[:, Hq:Hq + Hkv] += normal(Hkv, d)
        x = x.to(dt)
        parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["q"], s["k"], s["v"] = parts if c["fused"] else (p.contiguous() for p in parts)
        if c["rot"]:
            freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
            angle = torch.arange(c["cap"], device="cuda", dtype=torch.float64)[:, None] * freq
            s["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        else:
            s["rotary"] = None
        shape, kind = ((n_pages, Hkv, CHUNK * _row_bytes(c)), torch.uint8) if c["quant"] else ((n_pages, Hkv, CHUNK, d), dt)
        s["k_pages"], s["v_pages"] = (torch.zeros(shape, dtype=kind, device="cuda") for _ in range(2))
    else:
        if c["op"] == "decode4":
            s["q"] = normal(B, Hq, d).to(dt)
            near = torch.nn.functional.normalize(s["q"].float().unflatten(1, (Hkv, -1)).mean(2), dim=-1)   # [B, Hkv, d]
            owner = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
            owner[s["table"].flatten().long()] = torch.arange(B * nc, device="cuda") // nc
        lq_page = normal(n_pages, Hkv, d).to(dt)
        for name in ("k_pages", "v_pages")[: 1 if c["op"] == "summary" else 2]:
            blocks, summ = [], []
            per = max(1, (1 << 25) // (Hkv * CHUNK * d))
            for p in range(0, n_pages, per):
                m = min(per, n_pages - p)
                x = normal(m, Hkv, CHUNK, d)
                if name == "k_pages" and c["op"] == "decode4":   # one chunk in 64 is what the queries look for
                    hit = torch.rand(m, device="cuda", generator=gen) < 1 / 64
                    x += (1.5 * hit[:, None, None] * near[owner[p:p + m]])[:, :, None]
                if c["quant"]:
                    a, b = _pack_row(x)
                    x = torch.cat([a.flatten(-2), b.flatten(-2)], -1)
                else:
                    x = x.to(dt)
                blocks.append(x)
                if name == "k_pages" and c["op"] == "decode4":
                    summ.append(_summary(_unpack_block(x, d, torch.float32), lq_page[p:p + m].float()))
            s[name] = torch.cat(blocks)
            if summ:
                kp, bp = (torch.cat(v)[s["table"].long()].transpose(1, 2).contiguous() for v in zip(*summ))
                s["kprime"], s["bprime"], s["kmma"] = kp, bp, _operand(kp, bp) if c["dtype"] == "bf16" else None
        s["lq"] = lq_page[s["table"].long()].transpose(1, 2).contiguous()         # [B, Hkv, nc, d]
        if c["op"] == "summary":
            s["kprime"] = torch.zeros((B, Hkv, nc, d), device="cuda")
            s["bprime"] = torch.zeros((B, Hkv, nc), device="cuda")
            s["kmma"] = torch.zeros((B, Hkv, nc, d + EXT), dtype=torch.bfloat16, device="cuda") if c["dtype"] == "bf16" else None
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    return {"append": _append, "append4": _append4, "read4": _read4, "summary": _summary_step, "decode4": _decode4}[c["op"]](s)


def _run_own(s):
    from chunk_wise_sparse_b200 import hils

    c = s["case"]
    if c["op"].startswith("append"):
        rotary = None if s["rotary"] is None else hils.Rotary(s["rotary"], interleaved=c["interleaved"])
        q = hils.kv_append(s["k_pages"], s["v_pages"], s["table"], s["k"], s["v"], s["seqlens"], cu_tokens=s["cu"],
                           rotary=rotary, q=s["q"])
        if c["op"] == "append":
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        k, v = hils.kv_read(s["k_pages"], s["v_pages"], s["table"], s["seqlens"], s["T"], s["dtype"], cu_tokens=s["cu"])
        return {"q": q, "k": k, "v": v}
    if c["op"] == "read4":
        k, v = hils.kv_read(s["k_pages"], s["v_pages"], s["table"], s["seqlens"], s["T"], s["dtype"], cu_tokens=s["cu"])
        return {"k": k, "v": v}
    if c["op"] == "summary":
        summ = hils.Summary.of(s["kprime"], s["bprime"], s["kmma"])
        hils.landmark_summary_append(s["k_pages"], s["table"], s["lq"], s["seqlens"], s["T"], summ, cu_tokens=s["cu"])
        return {"kprime": s["kprime"], "bprime": s["bprime"], "kmma": s["kmma"]}
    summ = hils.Summary.of(s["kprime"], s["bprime"], s["kmma"])
    o, _, _ = hils.decode_step_quant(s["q"], s["k_pages"], s["v_pages"], s["table"], summ, s["seqlens"], c["K"],
                                     window=c["window"])
    return {"o": o}


def _places(s):
    """(sequence, position) of every new token."""
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    return b, s["seqlens"].long()[b] - (s["cu"].long()[b + 1] - t)


def _rotate(x, table, pos, interleaved):
    """x [T, H, d] rotated by the angles of each token's position, in 64 bits."""
    x = x.double()
    if table is None:
        return x
    cos, sin = table[pos].double()[:, None].chunk(2, -1)
    r = table.shape[1]
    a, b = (x[..., :r:2], x[..., 1:r:2]) if interleaved else (x[..., : r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), x[..., r:]], -1)


def _append(s):
    b, pos = _places(s)
    page, row = s["table"][b, pos // CHUNK].long(), pos % CHUNK
    il = s["case"]["interleaved"]
    s["k_pages"][page, :, row] = _rotate(s["k"], s["rotary"], pos, il).to(s["dtype"])
    s["v_pages"][page, :, row] = s["v"]
    return {"q": _rotate(s["q"], s["rotary"], pos, il).to(s["dtype"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _append4(s):
    b, pos = _places(s)
    page, row = s["table"][b, pos // CHUNK].long(), pos % CHUNK
    d, il = s["case"]["d"], s["case"]["interleaved"]
    n = CHUNK * d // 2
    for pages, x in ((s["k_pages"], _rotate(s["k"], s["rotary"], pos, il)), (s["v_pages"], s["v"].double())):
        codes, pairs = _pack_row(x)    # in 64 bits: a value next to the border of two codes takes the nearer one
        pages[..., :n].unflatten(-1, (CHUNK, d // 2))[page, :, row] = codes
        pages[..., n:].unflatten(-1, (CHUNK, d // 8))[page, :, row] = pairs
    return {"q": _rotate(s["q"], s["rotary"], pos, il).to(s["dtype"]), **_read4(s)}


def _read4(s):
    b, pos = _places(s)
    page, row = s["table"][b, pos // CHUNK].long(), pos % CHUNK
    d, got = s["case"]["d"], {}
    n = CHUNK * d // 2
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        codes = pages[..., :n].unflatten(-1, (CHUNK, 8, d // GROUP, 2))[page, :, row]            # [T, Hkv, e, g, 2]
        pairs = pages[..., n:].unflatten(-1, (CHUNK, d // 8))[page, :, row]
        pairs = pairs.view(torch.float16).unflatten(-1, (-1, 2)).float()
        q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).transpose(-3, -2).flatten(-2)  # [T, Hkv, g, 32]
        got[name] = (pairs[..., 1:] + pairs[..., :1] * q).flatten(-2).to(s["dtype"])
    return got


def _summary(k, lq):
    """k' and b' of keys [..., 64, d] under landmark queries [..., d]."""
    z = (k * lq[..., None, :]).sum(-1) / math.sqrt(k.shape[-1])
    p = z.softmax(-1)
    return (p[..., None] * k).sum(-2), z.logsumexp(-1) - (p * z).sum(-1)


def _operand(kp, bp):
    """The bf16 scoring operand: k', then b' / tau as the sum of two bf16 values, then zeros."""
    x = bp * math.sqrt(kp.shape[-1])
    hi = x.bfloat16()
    ext = torch.zeros((*bp.shape, EXT), dtype=torch.bfloat16, device=bp.device)
    ext[..., 0], ext[..., 1] = hi, (x - hi.float()).bfloat16()
    return torch.cat([kp.bfloat16(), ext], -1)


def _summary_step(s):
    c = s["case"]
    b, pos = _places(s)
    done = (pos % CHUNK == CHUNK - 1).nonzero().flatten()
    b, ch = b[done], pos[done] // CHUNK
    k = s["k_pages"][s["table"][b, ch].long()]
    k = _unpack_block(k, c["d"], torch.float32) if c["quant"] else k.float()
    kp, bp = _summary(k, s["lq"][b, :, ch].float())
    s["kprime"][b, :, ch], s["bprime"][b, :, ch] = kp, bp
    if s["kmma"] is not None:
        s["kmma"][b, :, ch] = _operand(kp, bp)
    return {"kprime": s["kprime"], "bprime": s["bprime"], "kmma": s["kmma"]}


def _decode4(s):
    c = s["case"]
    B, Hq, Hkv, d, K = c["B"], c["Hq"], c["Hkv"], c["d"], c["K"]
    G, wc, tau = Hq // Hkv, max(1, c["window"] // CHUNK), 1 / math.sqrt(d)
    q = s["q"].float().unflatten(1, (Hkv, G))
    chunk = (s["seqlens"].long() - 1) // CHUNK
    # the chunk scores, in 64 bits: the K-th and the next may lie close together
    if s["kmma"] is not None:
        score = torch.einsum("bhgd,bhcd->bhgc", q.double(), s["kmma"][..., :d].double())
        score = tau * (score + s["kmma"][:, :, None, :, d:d + 2].double().sum(-1))
    else:
        score = tau * torch.einsum("bhgd,bhcd->bhgc", q.double(), s["kprime"].double()) + s["bprime"][:, :, None].double()
    nc = score.shape[-1]
    score = score.masked_fill(torch.arange(nc, device="cuda") >= (chunk - wc + 1).view(B, 1, 1, 1), -math.inf)
    score, ids = score.sort(dim=-1, descending=True, stable=True)
    score, ids = score[..., :K].float(), ids[..., :K]
    near = chunk[:, None] - torch.arange(wc, device="cuda")                                     # the window's chunks
    at, h = torch.arange(B, device="cuda").view(B, 1, 1, 1), torch.arange(Hkv, device="cuda").view(1, Hkv, 1, 1)
    page = s["table"][at, ids].long()
    k, v = (_unpack_block(s[n][page, h], d, torch.float32) for n in ("k_pages", "v_pages"))   # [B, Hkv, G, K, 64, d]
    z = tau * torch.einsum("bhgd,bhgkjd->bhgkj", q, k)
    each = torch.einsum("bhgkj,bhgkjd->bhgkd", z.softmax(-1), v)
    page = s["table"][at, near.clamp(min=0).view(B, 1, 1, wc)].long()
    k, v = (_unpack_block(s[n][page, h], d, torch.float32).flatten(3, 4)[:, :, 0] for n in ("k_pages", "v_pages"))
    pos = near[:, :, None] * CHUNK + torch.arange(CHUNK, device="cuda")
    seen = ((pos >= 0) & (pos < s["seqlens"].view(B, 1, 1))).flatten(1).view(B, 1, 1, -1)
    z = (tau * torch.einsum("bhgd,bhjd->bhgj", q, k)).masked_fill(~seen, -math.inf)
    local = torch.einsum("bhgj,bhjd->bhgd", z.softmax(-1), v.masked_fill(~seen[:, 0, 0][:, None, :, None], 0))
    w = torch.cat([score, z.logsumexp(-1, keepdim=True)], -1).softmax(-1)
    o = torch.einsum("bhgk,bhgkd->bhgd", w[..., :-1], each) + w[..., -1:] * local
    return {"o": o.flatten(1, 2).to(s["dtype"])}


# ---------------------------------------------------------------- the same from the definitions, in 64 bits

def _held(x):
    """What a 4-bit cache holds of x [..., d], in 64 bits, value by value."""
    d = x.shape[-1]
    out = torch.empty_like(x)
    for g in range(0, d, GROUP):
        y = x[..., g:g + GROUP]
        low = y.min(-1, keepdim=True).values
        step = ((y.max(-1, keepdim=True).values - low) / 15).to(torch.float16).double()
        low = low.to(torch.float16).double()
        code = torch.nan_to_num((y - low) / step, 0.0, 0.0, 0.0).round().clamp(0, 15)
        out[..., g:g + GROUP] = low + step * code
    return out


def _values(block, d):
    """The 64 rows of blocks [..., bytes] in 64 bits, each dim from its own place."""
    rows = block[..., : CHUNK * d // 2].reshape(*block.shape[:-1], CHUNK, d // 2).to(torch.int32)
    pairs = block[..., CHUNK * d // 2:].contiguous().view(torch.float16).double().reshape(*block.shape[:-1], CHUNK, d // GROUP, 2)
    i = torch.arange(d, device=block.device)
    g, e, nib = i // GROUP, i % GROUP // 4, i % 4
    byte = 2 * (e * (d // GROUP) + g) + nib // 2
    code = (rows[..., byte] >> (4 * (nib % 2))) & 15
    return pairs[..., g, 1] + pairs[..., g, 0] * code.double()


def _turned(x, table, first, interleaved):
    """x [n, H, d] of the positions first .. first + n - 1, rotated as complex numbers."""
    y = x.double().clone()
    if table is None:
        return y
    r, t = table.shape[1], table[first:first + len(x)].double()
    turn = torch.complex(t[:, : r // 2], t[:, r // 2:])[:, None]
    if interleaved:
        y[..., :r] = torch.view_as_real(torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], -1, 2)) * turn).flatten(-2)
    else:
        w = torch.complex(y[..., : r // 2], y[..., r // 2:r]) * turn
        y[..., :r] = torch.cat([w.real, w.imag], -1)
    return y


def exact(c, seed):
    s = prepare(c, seed)
    d, Hkv, table = c["d"], c["Hkv"], s["table"].long()
    batch, cu, il = _batch(c), s["cu"].tolist(), c["interleaved"]
    if c["op"].startswith("append"):
        q = torch.cat([_turned(s["q"][cu[b]:cu[b + 1]], s["rotary"], a, il) for b, (a, _) in enumerate(batch)])
        k = torch.cat([_turned(s["k"][cu[b]:cu[b + 1]], s["rotary"], a, il) for b, (a, _) in enumerate(batch)])
        v = s["v"].double()
        if c["op"] == "append4":
            return {"q": q, "k": _held(k), "v": _held(v)}
        out = {"q": q}
        for name, x in (("k_pages", k), ("v_pages", v)):
            pool = torch.zeros((s["n_pages"], CHUNK, Hkv, d), dtype=torch.float64, device="cuda")
            for b, (a, n) in enumerate(batch):
                p = torch.arange(a, a + n, device="cuda")
                pool.view(-1, Hkv, d)[table[b][p // CHUNK] * CHUNK + p % CHUNK] = x[cu[b]:cu[b + 1]]
            out[name] = pool.transpose(1, 2)
        return out
    if c["op"] == "read4":
        out = {}
        for name in ("k", "v"):
            rows = []
            for b, (a, n) in enumerate(batch):
                pages = table[b, a // CHUNK:(a + n - 1) // CHUNK + 1]
                x = _values(s[name + "_pages"][pages], d).transpose(1, 2).reshape(-1, Hkv, d)
                rows.append(x[a % CHUNK:a % CHUNK + n].to(torch.float32 if c["dtype"] == "bf16" else torch.float64))
            out[name] = torch.cat(rows)
        return {n: x.double() for n, x in out.items()}
    root = math.sqrt(d)
    if c["op"] == "summary":
        kp, bp = s["kprime"].double(), s["bprime"].double()
        mma = torch.zeros((*bp.shape, d + EXT), dtype=torch.float64, device="cuda")
        for b, (a, n) in enumerate(batch):
            lo, hi = a // CHUNK, (a + n) // CHUNK
            for at in range(lo, hi, 128):
                ch = torch.arange(at, min(hi, at + 128), device="cuda")
                block = s["k_pages"][table[b, ch]].transpose(0, 1)                        # [Hkv, chunks, ...]
                k = _values(block, d) if c["quant"] else block.double()
                z = torch.einsum("hcjd,hcd->hcj", k, s["lq"][b, :, ch].double()) / root
                p = torch.exp(z - z.max(-1, keepdim=True).values)
                p /= p.sum(-1, keepdim=True)
                kp[b, :, ch] = torch.einsum("hcj,hcjd->hcd", p, k)
                bp[b, :, ch] = -torch.special.xlogy(p, p).sum(-1)
        if s["kmma"] is None:
            return {"kprime": kp, "bprime": bp, "kmma": None}
        mma[..., :d] = kp
        mma[..., d] = (bp * root).to(torch.bfloat16).double()
        mma[..., d + 1] = bp * root - mma[..., d]
        return {"kprime": kp, "bprime": bp, "kmma": mma}
    # decode4, row by row
    G, wc = c["Hq"] // Hkv, max(1, c["window"] // CHUNK)
    o = torch.empty((c["B"], c["Hq"], d), dtype=torch.float64, device="cuda")
    for b, (last, _) in enumerate(batch):
        chunk = last // CHUNK
        cand, first = max(0, chunk - wc + 1), max(0, chunk - wc + 1)
        for hq in range(c["Hq"]):
            h, q = hq // G, s["q"][b, hq].double()
            if s["kmma"] is not None:
                m = s["kmma"][b, h, :cand].double()
                score = (m[:, :d] @ q + m[:, d] + m[:, d + 1]) / root
            else:
                score = s["kprime"][b, h, :cand].double() @ q / root + s["bprime"][b, h, :cand].double()
            keep = torch.argsort(score, descending=True, stable=True)[: c["K"]]
            kept = s["k_pages"][table[b, keep], h], s["v_pages"][table[b, keep], h]
            k, v = (_values(x, d) for x in kept)
            p = torch.exp(k @ q / root)
            each = torch.einsum("cj,cjd->cd", p / p.sum(-1, keepdim=True), v)
            near = torch.arange(first, chunk + 1, device="cuda")
            k, v = (_values(s[n][table[b, near], h], d).reshape(-1, d)[: last + 1 - first * CHUNK] for n in ("k_pages", "v_pages"))
            p = torch.exp(k @ q / root)
            w = torch.exp(score[keep])
            o[b, hq] = (w @ each + p @ v) / (w.sum() + p.sum())   # the window's weight is the exponential of its log-sum-exp
    return {"o": o}
