"""What is measured of the serving operators beside the sparse attention: rotary
positions, appending keys and values to a paged cache, and the attention of new
tokens over that cache (with the documents selected for a query, if any).

Where `own` is false the operators run in their plain form, elementary torch
operations in 32 bits rounded once at the end; where it is true they run as a
user's program calls them in this library.
"""
import math
import random

import torch

own = False  # set from outside: the library's kernels, or the plain forms

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA = 1e6  # the base of this repository's workloads
PAGES = (8, 16, 32, 64, 128, 256)


# --------------------------------------------------------------------------- cases
def listed():
    """Head counts are those of this repository's workloads (32 query heads over 8 KV heads of
    128, 4 over 2 of 64) unless a case is there for another grouping."""
    return [
        # one decoding step's queries and keys of a single request: the latency of a call
        dict(name="rope_token", op="rope", dtype="bf16", N=1, H=40, Hall=48, d=128, rd=128, layout="half", back=False,
             max_len=4096),
        # a prompt's queries and keys, rotated where the fused projection left them
        dict(name="rope_prompt", op="rope", dtype="bf16", N=4096, H=40, Hall=48, d=128, rd=128, layout="half",
             back=False, max_len=16384),
        # the gradient of a rotation of a quarter of each head, fp32 as a training step keeps it
        dict(name="rope_grad", op="rope", dtype="f32", N=6001, H=40, Hall=40, d=128, rd=32, layout="interleaved",
             back=True, max_len=16384),
        # a decoding step of 64 requests: one token each, into pages of 16
        dict(name="append_tokens", op="append", dtype="bf16", B=64, chunks=0, q_lo=1, q_hi=1, ctx_lo=100, ctx_hi=1500,
             Hq=32, Hkv=8, d=128, rd=128, layout="half", page=16, lens=1),
        # six prompts at once, half of each head rotated, pages of 64
        dict(name="append_prompts", op="append", dtype="bf16", B=6, chunks=6, q_lo=700, q_hi=2600, ctx_lo=0, ctx_hi=900,
             Hq=32, Hkv=8, d=128, rd=64, layout="interleaved", page=64, lens=2),
        # one request's next token over a short history: the latency of a call
        dict(name="attn_token", op="attn", dtype="bf16", B=1, chunks=0, q_lo=1, q_hi=1, ctx_lo=1000, ctx_hi=1000, Hq=32,
             Hkv=8, d=128, page=16, k=0, docs=0, rows=0, lens=3),
        # 64 requests' next tokens over their selected documents and some 4096 local tokens
        dict(name="attn_tokens_memory", op="attn", dtype="bf16", B=64, chunks=0, q_lo=1, q_hi=1, ctx_lo=3500,
             ctx_hi=4700, Hq=32, Hkv=8, d=128, page=64, k=16, docs=512, rows=8, lens=4),
        # three drafted tokens of a few long conversations
        dict(name="attn_drafts_long", op="attn", dtype="bf16", B=5, chunks=5, q_lo=3, q_hi=3, ctx_lo=20000,
             ctx_hi=131000, Hq=32, Hkv=8, d=128, page=128, k=0, docs=0, rows=0, lens=5),
        # a question of 512 tokens over its selected documents and some context
        dict(name="attn_chunk_memory", op="attn", dtype="bf16", B=1, chunks=1, q_lo=512, q_hi=512, ctx_lo=1500,
             ctx_hi=1500, Hq=32, Hkv=8, d=128, page=16, k=16, docs=512, rows=8, lens=6),
        # one part of a long prompt over what was cached before
        dict(name="attn_chunk_long", op="attn", dtype="bf16", B=1, chunks=1, q_lo=4096, q_hi=4096, ctx_lo=28000,
             ctx_hi=28000, Hq=32, Hkv=8, d=128, page=256, k=0, docs=0, rows=0, lens=7),
        # a serving batch: a few parts of prompts among single tokens, small heads, 5 query heads a KV head
        dict(name="attn_mixed", op="attn", dtype="bf16", B=23, chunks=4, q_lo=90, q_hi=700, ctx_lo=0, ctx_hi=6000,
             Hq=40, Hkv=8, d=64, page=32, k=0, docs=0, rows=0, lens=8),
        # the small fp32 configuration: a short question over two documents and its context
        dict(name="attn_f32", op="attn", dtype="f32", B=3, chunks=3, q_lo=20, q_hi=75, ctx_lo=200, ctx_hi=900, Hq=4,
             Hkv=2, d=64, page=8, k=2, docs=64, rows=8, lens=9),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        H = rng.randint(1, 64)
        N = _log(rng, 1, max(1, min(32768, 60_000_000 // (H * d))))
        return dict(op=op, dtype=dtype, N=N, H=H, Hall=H + rng.choice([0, 8]), d=d, rd=rng.choice([d // 4, d // 2, d]),
                    layout=layout, back=rng.random() < 0.5, max_len=_log(rng, 64, 65536))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice(PAGES)
    if op == "append":
        B = _log(rng, 1, 128)
        chunks = rng.choice([0, rng.randint(0, min(B, 8))])
        q_hi = _log(rng, 1, 2000)
        ctx = _log(rng, 1, 2000)
        return dict(op=op, dtype=dtype, B=B, chunks=chunks, q_lo=max(1, q_hi // 3), q_hi=q_hi, ctx_lo=ctx // 4,
                    ctx_hi=ctx, Hq=Hkv * G, Hkv=Hkv, d=d, rd=rng.choice([d // 4, d // 2, d]), layout=layout, page=page,
                    lens=rng.randint(1, 1 << 30))
    k = rng.choice([0, 0, 2, 16])
    rows = rng.randint(1, 12)
    kind = rng.choice(["tokens", "drafts", "chunks", "mixed"])
    if kind in ("tokens", "drafts"):
        B = _log(rng, 1, 100)
        q_lo, q_hi = (1, 1) if kind == "tokens" else (1, rng.randint(2, 5))
        chunks = 0 if kind == "tokens" else B
        top = 3_000_000 // (B * Hkv * (2 if dtype == "f32" else 1))
        ctx = _log(rng, 1, max(1, min(100_000, top)))
    else:
        B = rng.randint(1, 4) if kind == "chunks" else rng.randint(2, 40)
        chunks = B if kind == "chunks" else min(B, rng.randint(1, 3))
        q_hi = _log(rng, 6, 1500)
        q_lo = max(2, q_hi // 2)
        ctx = _log(rng, 1, 12_000)
        if dtype == "f32":
            q_hi, q_lo, ctx = min(q_hi, 600), min(q_lo, 300), min(ctx, 4000)
    return dict(op=op, dtype=dtype, B=B, chunks=chunks, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx // 3, ctx_hi=ctx, Hq=Hkv * G,
                Hkv=Hkv, d=d, page=page, k=k, docs=64 if k else 0, rows=rows if k else 0, lens=rng.randint(1, 1 << 30))


def _lengths(case):
    """New tokens and earlier tokens of every sequence; the longer parts come first."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) if b < case["chunks"] else 1 for b in range(case["B"])]
    return q, [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in q]


# --------------------------------------------------------------------------- inputs
def _table(rd, max_len):
    """fp32 (cos, sin) of p * theta^(-2 i / rd), from angles in 64 bits: [max_len, rd / 2, 2]."""
    i = torch.arange(rd // 2, dtype=torch.float64, device=DEV)
    ang = torch.arange(max_len, dtype=torch.float64, device=DEV)[:, None] * THETA ** (-2.0 * i / rd)
    return torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    d = case["d"]

    def normal(*shape):
        return (0.5 * torch.randn(shape, generator=gen, device=DEV)).to(dt)

    s = dict(case=case)
    if case["op"] == "rope":
        N, H = case["N"], case["H"]
        s["x"] = normal(N, case["Hall"], d)[:, :H]  # the rotated heads of a fused projection
        s["pos"] = torch.randint(0, case["max_len"], (N,), generator=gen, device=DEV, dtype=torch.int32)
        s["cs"] = _table(case["rd"], case["max_len"])
        s["out"] = torch.empty((N, H, d), dtype=dt, device=DEV)
        return s

    q_len, ctx = _lengths(case)
    B, Hq, Hkv, page = case["B"], case["Hq"], case["Hkv"], case["page"]
    N = sum(q_len)
    total = [a + b for a, b in zip(q_len, ctx)]
    per_seq = [-(-t // page) for t in total]
    pages = sum(per_seq) + 7  # some of the pool's pages belong to nobody
    off = [0]
    for n in q_len:
        off.append(off[-1] + n)
    s["q_off"] = torch.tensor(off, dtype=torch.int64, device=DEV)
    s["seq_len"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    s["max_q"] = max(q_len)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    width = max(per_seq)
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)  # entries past a sequence's pages are unused
    at = 0
    for b, n in enumerate(per_seq):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["K"], s["V"] = normal(pages, page, Hkv, d), normal(pages, page, Hkv, d)
    if case["op"] == "append":
        qkv = normal(N, Hq + 2 * Hkv, d)  # one fused projection
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["cs"] = _table(case["rd"], max(total))
        s["q_out"] = torch.empty((N, Hq, d), dtype=dt, device=DEV)
        return s
    s["q"] = normal(N, Hq, d)
    s["O"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((Hq, N), dtype=torch.float32, device=DEV)
    k, rows, docs = case["k"], case["rows"], case["docs"]
    s["idx"] = s["chunk_off"] = s["Kbar"] = s["Vbar"] = None
    if k:
        s["idx"] = torch.rand((B, docs), generator=gen, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
        s["chunk_off"] = rows * torch.arange(docs + 1, dtype=torch.int64, device=DEV)
        s["Kbar"], s["Vbar"] = normal(docs * rows, Hkv, d), normal(docs * rows, Hkv, d)
    if own:
        import routed_sparse_attention_chunk_b200 as msa
        n = msa.paged_attn_workspace_size(s["q"].dtype, B, s["max_q"], Hq, Hkv, d, k, k * rows)
        s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "rope":
        x = s["x"].float()
        return _rotate(x, s["cs"][s["pos"].long()], case["layout"], case["back"]).to(s["x"].dtype)
    if case["op"] == "append":
        return _plain_append(s, case)
    return _plain_attn(s, case)


def _run_own(s, case):
    import routed_sparse_attention_chunk_b200 as msa
    if case["op"] == "rope":
        layout = msa.ROPE_HALF if case["layout"] == "half" else msa.ROPE_INTERLEAVED
        f = msa.rope_backward if case["back"] else msa.rope
        f(s["x"], s["pos"], s["cs"], s["out"], layout=layout)
        return s["out"]
    if case["op"] == "append":
        layout = msa.ROPE_HALF if case["layout"] == "half" else msa.ROPE_INTERLEAVED
        msa.paged_append(s["q"], s["k"], s["v"], s["q_off"], s["seq_len"], s["table"], s["K"], s["V"],
                         rope_cs=s["cs"], q_out=s["q_out"], layout=layout)
        return s["q_out"], s["K"], s["V"]
    msa.paged_attn(s["q"], s["q_off"], s["max_q"], s["K"], s["V"], s["table"], s["seq_len"], s["O"], s["ws"],
                   lse=s["lse"], topk_idx=s["idx"], doc_chunk_off=s["chunk_off"], Kbar=s["Kbar"], Vbar=s["Vbar"],
                   Mmax=case["k"] * case["rows"])
    return s["O"], s["lse"]


def _rotate(x, cs, layout, back):
    """x [n, H, d] in 32 bits, cs [n, rd / 2, 2]: the first rd dimensions of every head rotated
    (or, for the gradient, by the transposed rotation)."""
    c, w = cs[:, None, :, 0], cs[:, None, :, 1]
    if back:
        w = -w
    rd = 2 * c.shape[-1]
    if layout == "half":
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat([a * c - b * w, a * w + b * c], -1)
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack([a * c - b * w, a * w + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def _positions(s, case):
    """Owning sequence and cache position of every new token."""
    n = s["q_off"][1:] - s["q_off"][:-1]
    seq = torch.repeat_interleave(torch.arange(case["B"], device=DEV), n, output_size=s["q"].shape[0])
    i = torch.arange(s["q"].shape[0], device=DEV) - s["q_off"][seq]
    return seq, s["seq_len"][seq].long() - n[seq] + i


def _plain_append(s, case):
    seq, pos = _positions(s, case)
    cs = s["cs"][pos]
    q = _rotate(s["q"].float(), cs, case["layout"], False).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cs, case["layout"], False).to(s["k"].dtype)
    page, row = s["table"][seq, pos // case["page"]].long(), pos % case["page"]
    s["K"][page, row] = k
    s["V"][page, row] = s["v"]
    return q, s["K"], s["V"]


def _plain_attn(s, case):
    q_len, ctx = _lengths(case)
    Hkv, G, d, page = case["Hkv"], case["Hq"] // case["Hkv"], case["d"], case["page"]
    out, lses, at = [], [], 0
    for b, (n, c) in enumerate(zip(q_len, ctx)):
        ids = s["table"][b, :-(-(n + c) // page)].long()
        K = s["K"][ids].flatten(0, 1)[:n + c].float()
        V = s["V"][ids].flatten(0, 1)[:n + c].float()
        m = 0
        if case["k"]:
            rows = (s["idx"][b].long()[:, None] * case["rows"] + torch.arange(case["rows"], device=DEV)).flatten()
            K = torch.cat([s["Kbar"][rows].float(), K])
            V = torch.cat([s["Vbar"][rows].float(), V])
            m = rows.numel()
        q = s["q"][at:at + n].float().view(n, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, n * G, d)
        K, V = K.transpose(0, 1), V.transpose(0, 1)  # [Hkv, keys, d]
        # key j of the local ones is seen by token i where j <= c + i
        hide = torch.arange(n + c + m, device=DEV)[None] > m + c + torch.arange(n, device=DEV)[:, None]
        step = max(1, (1 << 29) // (n * G * (n + c + m)))  # KV heads at a time: a long chunk's scores are large
        o_b, l_b = [], []
        for h in range(0, Hkv, step):
            sc = (q[h:h + step] @ K[h:h + step].mT * d ** -0.5).unflatten(1, (n, G))
            sc.masked_fill_(hide[:, None], float("-inf"))
            top = sc.amax(-1, keepdim=True)
            p = sc.sub_(top).exp_()
            z = p.sum(-1, keepdim=True)
            o_b.append((p.flatten(1, 2) @ V[h:h + step]).unflatten(1, (n, G)) / z)
            l_b.append((top + z.log())[..., 0])
        out.append(torch.cat(o_b).transpose(0, 1).flatten(1, 2).to(s["q"].dtype))
        lses.append(torch.cat(l_b).transpose(1, 2).flatten(0, 1))
        at += n
    return torch.cat(out), torch.cat(lses, 1)


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s["x"], s["pos"].long(), s["cs"], case)
    if case["op"] == "append":
        K, V, at = s["K"].double(), s["V"].double(), 0
        pos = []
        for b, (n, c) in enumerate(zip(*_lengths(case))):
            p = torch.arange(c, c + n, device=DEV)
            slot = s["table"][b].long()[p // case["page"]] * case["page"] + p % case["page"]
            K.view(-1, *K.shape[2:])[slot] = _exact_rotation(s["k"][at:at + n], p, s["cs"], case)
            V.view(-1, *V.shape[2:])[slot] = s["v"][at:at + n].double()
            pos.append(p)
            at += n
        return _exact_rotation(s["q"], torch.cat(pos), s["cs"], case), K, V
    return _exact_attn(s, case)


def _exact_rotation(x, pos, cs, case):
    """Pairs as complex numbers times the table's cos + i sin (its conjugate for the gradient)."""
    turn = torch.view_as_complex(cs.double())[pos][:, None]
    if case.get("back"):
        turn = turn.conj()
    y, rd = x.double().clone(), case["rd"]
    h = rd // 2
    first, second = (slice(0, h), slice(h, rd)) if case["layout"] == "half" else (slice(0, rd, 2), slice(1, rd, 2))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_attn(s, case):
    d, G = case["d"], case["Hq"] // case["Hkv"]
    O = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    off = s["q_off"].tolist()
    for b, length in enumerate(s["seq_len"].tolist()):
        j = torch.arange(length, device=DEV)
        slot = s["table"][b].long()[j // case["page"]] * case["page"] + j % case["page"]
        i = torch.arange(off[b], off[b + 1], device=DEV)
        first_pos = length - (off[b + 1] - off[b])
        for h in range(case["Hq"]):
            g = h // G
            k, v = s["K"][:, :, g].reshape(-1, d)[slot].double(), s["V"][:, :, g].reshape(-1, d)[slot].double()
            seen = j[None] <= (first_pos + i - off[b])[:, None]
            if case["k"]:
                docs = s["idx"][b].tolist()
                bounds = s["chunk_off"].tolist()
                rows = torch.tensor([c for t in docs for c in range(bounds[t], bounds[t + 1])], device=DEV)
                k, v = torch.cat([s["Kbar"][rows, g].double(), k]), torch.cat([s["Vbar"][rows, g].double(), v])
                seen = torch.cat([seen.new_ones(len(i), len(rows)), seen], 1)
            score = torch.where(seen, s["q"][i, h].double() @ k.T / math.sqrt(d), -math.inf)
            l = torch.logsumexp(score, 1)
            lse[h, i] = l
            O[i, h] = torch.exp(score - l[:, None]) @ v
    return O, lse


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "rope":
        rows = min(case["N"], case["max_len"])
        return {"bytes": 2 * case["N"] * case["H"] * d * e + 4 * case["N"] + rows * case["rd"] * 4,
                "flops": 3 * case["N"] * case["H"] * case["rd"]}
    q_len, ctx = _lengths(case)
    N, total = sum(q_len), sum(q_len) + sum(ctx)
    Hq, Hkv = case["Hq"], case["Hkv"]
    meta = 8 * (case["B"] + 1) + 4 * case["B"]
    if case["op"] == "append":
        return {"bytes": 2 * N * (Hq + 2 * Hkv) * d * e + N * case["rd"] * 4 + 4 * N + meta,
                "flops": 3 * N * (Hq + Hkv) * case["rd"]}
    mem = case["k"] * case["rows"]
    pairs = sum(n * (c + mem) + n * (n + 1) // 2 for n, c in zip(q_len, ctx))
    # a bank row that several requests selected counts once for each of them, up to the whole bank
    bank = min(mem * case["B"], case["docs"] * case["rows"])
    return {"bytes": 2 * N * Hq * d * e + 4 * N * Hq + 2 * (total + bank) * Hkv * d * e + 4 * (total // case["page"])
            + 4 * case["B"] * case["k"] + meta,
            "flops": 4 * pairs * Hq * d}
