"""What is measured of the operators in front of sparse attention: the quantised index cache (written and
read back), the cheap score of every cached token or block, the selection of the best blocks, and the
attention over the selected pages.

Where ``own`` is false ``run`` computes the plain form with elementary torch operations; where it is true it
calls the framework.
"""
import math

import torch

own = False

DEV = "cuda"
D = 128                     # width of an index key
NOPE = 64                   # its values before the rotated part
ENTRY = {"bf16": 1152, "fp8": 576, "fp8_ds_mla": 656}
NEG = float("-inf")


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a small batch: the index queries and keys of 32 tokens
        dict(name="insert_decode_fp8", op="insert", fmt="fp8", B=32, Hi=64, ps=64, rope=True),
        # a chunk of a long prefill, a ragged size
        dict(name="insert_prefill_fp8", op="insert", fmt="fp8", B=8191, Hi=64, ps=64, rope=True),
        # the cached keys of one short request read back
        dict(name="gather_short_fp8", op="gather", fmt="fp8", B=1, lo=1021, hi=1021, ps=64),
        # the cached context of a chunk of requests read back for a long prefill
        dict(name="gather_context_fp8", op="gather", fmt="fp8", B=13, lo=1024, hi=32768, ps=64),
        # token scores of a decode step over long contexts
        dict(name="scores_decode_fp8", op="scores", fmt="fp8", B=64, q=1, Hi=64, lo=16384, hi=131072, ps=64, bt=1),
        # block scores of speculative rows over short contexts, unquantised keys
        dict(name="scores_verify_blocks_bf16", op="scores", fmt="bf16", B=32, q=4, Hi=32, lo=1024, hi=8192, ps=64, bt=64),
        # token scores of a prefill chunk at the end of long contexts: bound by the products
        dict(name="scores_prefill_fp8", op="scores", fmt="fp8", B=2, q=2048, Hi=64, lo=20000, hi=32768, ps=64, bt=1),
        # top-2048 of every row of a decode step over long contexts, as cache slots
        dict(name="select_decode_slots", op="select", B=32, q=1, lo=16384, hi=131072, bt=1, k=2048, ps=64, first=0, last=0, slots=True, grain=0),
        # top-2048 of every row of a prefill chunk
        dict(name="select_prefill", op="select", B=1, q=4096, lo=65536, hi=65536, bt=1, k=2048, ps=64, first=0, last=0, slots=False, grain=0),
        # the best 32 pages of a decode step, the first and the newest always among them
        dict(name="select_blocks", op="select", B=128, q=1, lo=8192, hi=32768, bt=64, k=32, ps=64, first=1, last=2, slots=False, grain=0),
        # decode over 32 selected pages of a record cache, many heads
        dict(name="selected_decode_ds", op="selected", fmt="fp8_ds_mla", B=128, q=1, H=96, lo=8192, hi=32768, ps=64, k=32),
        # decode over 16 selected pages of a bf16 cache, few heads
        dict(name="selected_decode_bf16", op="selected", fmt="bf16", B=32, q=1, H=16, lo=1024, hi=8192, ps=64, k=16),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["insert", "gather", "scores", "scores", "select", "select", "selected"])
    ps = rng.choice([16, 32, 64, 128])
    if op == "insert":
        return dict(op=op, fmt=rng.choice(["fp8", "bf16"]), B=_spread(rng, 1, 8192), Hi=rng.randint(1, 64), ps=ps, rope=rng.random() < 0.8)
    if op == "gather":
        B = _spread(rng, 1, 32)
        hi = _spread(rng, 1, 200000 // B)
        return dict(op=op, fmt=rng.choice(["fp8", "bf16"]), B=B, lo=rng.randint(0, hi), hi=hi, ps=ps)
    if op == "scores":
        fmt, Hi = rng.choice(["fp8", "bf16"]), rng.choice([64, 32, rng.randint(1, 64)])
        bt = rng.choice([1, 1, 16, 32, 64, 128])
        if rng.random() < 0.6:      # decode and speculative rows
            B, q = _spread(rng, 1, 64), rng.choice([1, 1, 2, 4, rng.randint(1, 8)])
            hi = _spread(rng, 1, min(131072, 4000000 // (B * q)))
        else:                       # a prefill chunk
            B, q = rng.randint(1, 3), _spread(rng, 16, 1024)
            hi = _spread(rng, q, 16384)
        return dict(op=op, fmt=fmt, B=B, q=q, Hi=Hi, lo=rng.randint(max(1, hi // 2), hi), hi=hi, ps=ps, bt=bt)
    if op == "select":
        B, q = _spread(rng, 1, 64), rng.choice([1, 1, 4, _spread(rng, 1, 64)])
        bt = rng.choice([1, 1, 64])
        hi = _spread(rng, 1, min(262144, 30000000 // (B * q))) * bt
        k = _spread(rng, 1, 2048) if bt == 1 else _spread(rng, 1, 128)
        first = rng.choice([0, 0, min(k, 1)])
        last = rng.choice([0, 0, min(k - first, 2)])
        return dict(op=op, B=B, q=q, lo=rng.randint(1, hi), hi=hi, bt=bt, k=k, ps=ps, first=first, last=last, slots=rng.random() < 0.5, grain=rng.choice([0, 0, 4]))
    fmt = rng.choice(["bf16", "fp8", "fp8_ds_mla"])
    hi = _spread(rng, 1, 16384)
    q = rng.choice([1, 1, 1, 2, 4])
    return dict(op=op, fmt=fmt, B=_spread(rng, 1, 64), q=q, H=rng.choice([16, 16, 32, 64, 96, 128, rng.randint(1, 128)]), lo=rng.randint(1, hi), hi=hi, ps=ps, k=_spread(rng, 1, 1024 // ps))


# ------------------------------------------------------------------------------------------ shapes

def _lens(case):
    """Context lengths of the requests (the new tokens included), spread over [lo, hi]; the last one is hi."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    return [hi if b == B - 1 else lo + int((hi - lo) * math.modf((b + 1) * 0.6180339887498949)[0]) for b in range(B)]


def _rows(case):
    """Query rows of the requests: q each, but fewer where the context is shorter or in a ragged chunk."""
    L, q = _lens(case), case["q"]
    n = [q if q < 16 or b == 0 else max(1, q - 37 * b % q) for b in range(case["B"])]
    return [min(a, b) for a, b in zip(n, L)]


def _visible(case):
    """Visible tokens of every row, rows grouped by request."""
    return [L - n + i + 1 for L, n in zip(_lens(case), _rows(case)) for i in range(n)]


def work(case):
    op = case["op"]
    e = 2 if case.get("fmt") == "bf16" else 1
    if op == "insert":
        T, Hi, sc = case["B"], case["Hi"], 4 * (2 - e)
        rd = T * (Hi * (2 * D + 4) + 2 * D + 8) + (T * 264 if case["rope"] else 0)
        return {"bytes": rd + T * (Hi * (D * e + 4) + D * e + sc), "flops": T * (Hi + 1) * D * 4}
    if op == "gather":
        n = sum(_lens(case))
        return {"bytes": n * (D * e + 4 * (2 - e) + 2 * D), "flops": n * D}
    if op == "scores":
        vis, Hi = _visible(case), case["Hi"]
        keys = sum(_lens(case)) * (D * e + 4 * (2 - e))
        out = 4 * sum(-(-v // case["bt"]) for v in vis)
        return {"bytes": keys + len(vis) * Hi * (D * e + 4) + out, "flops": sum(vis) * Hi * (2 * D + 3)}
    if op == "select":
        vis = _visible(case)
        cols = sum(-(-v // case["bt"]) for v in vis)
        return {"bytes": 4 * cols + 4 * len(vis) * case["k"] * (1 + (case["bt"] if case["slots"] else 0)), "flops": cols}
    vis, H, ps = _visible(case), case["H"], case["ps"]
    toks = sum(min(v, case["k"] * ps) for v in vis)
    once = min(toks, sum(_lens(case)))
    eq = 1 if case["fmt"] == "fp8" else 2
    return {"bytes": once * ENTRY[case["fmt"]] + len(vis) * (H * (576 * eq + 1028) + 4 * case["k"]), "flops": toks * H * 2 * (576 + 512)}


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pow2_quant(x):
    """Codes and scale of the last dimension: scale 2^k, k least with amax <= 448 * 2^k."""
    amax = x.abs().amax(-1, keepdim=True)
    m, ex = torch.frexp(amax)
    k = torch.where(amax == 0, torch.zeros_like(ex), torch.where(m <= 0.875, ex - 9, ex - 8)).clamp(min=-126)
    return torch.ldexp(x, -k).to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(amax), k).squeeze(-1)


def _table(g, lens, ps, extra=3):
    """A shuffled block table for the lengths, and the number of blocks in the cache."""
    per = [-(-n // ps) for n in lens]
    nb = sum(per) + extra
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    w = max(1, max(per))
    start = torch.tensor([sum(per[:b]) for b in range(len(per))], device=DEV).unsqueeze(1)
    col = torch.arange(w, device=DEV).unsqueeze(0)
    have = col < torch.tensor(per, device=DEV).unsqueeze(1)
    return torch.where(have, ids[(start + col).clamp(max=nb - 1)], torch.zeros((), dtype=torch.int32, device=DEV)).contiguous(), nb


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _index_cache(g, nb, ps, fmt):
    x = torch.randn((nb, ps, D), generator=g, device=DEV)
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    x = x * torch.exp(torch.randn((nb, ps, 1), generator=g, device=DEV))
    codes, scale = _pow2_quant(x)
    return codes.view(torch.uint8), scale.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case}
    if op == "insert":
        T, Hi, ps = case["B"], case["Hi"], case["ps"]
        s["q"] = torch.randn((T, Hi, D), generator=g, device=DEV).to(torch.bfloat16)
        s["k"] = torch.randn((T, D), generator=g, device=DEV).to(torch.bfloat16)
        s["w"] = torch.randn((T, Hi), generator=g, device=DEV)
        s["weight_scale"] = float(D ** -0.5 * Hi ** -0.5)
        nb = -(-T // ps) + 2
        s["slots"] = torch.randperm(nb * ps, generator=g, device=DEV)[:T].contiguous()
        s["positions"] = s["cos_sin"] = None
        if case["rope"]:
            s["positions"] = torch.randint(0, 131072, (T,), generator=g, device=DEV)
            inv = 10000.0 ** (-torch.arange(0, 32, dtype=torch.float64, device=DEV) / 32)
            ang = torch.arange(131072, dtype=torch.float64, device=DEV).unsqueeze(1) * inv
            s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["cache"], s["scales"] = _index_cache(g, nb, ps, case["fmt"])
        return s
    lens = _lens(case)
    ps = case["ps"]
    s["table"], nb = _table(g, lens, ps)
    s["seq_lens"] = _i32(lens)
    if op == "gather":
        s["cache"], s["scales"] = _index_cache(g, nb, ps, case["fmt"])
        s["cu"] = _i32(_cum(lens))
        s["n"] = sum(lens)
        return s
    rows = _rows(case)
    T = sum(rows)
    s["cu_q"] = _i32(_cum(rows))
    if op == "scores":
        Hi = case["Hi"]
        s["cache"], s["scales"] = _index_cache(g, nb, ps, case["fmt"])
        q = torch.randn((T, Hi, D), generator=g, device=DEV)
        w = torch.rand((T, Hi), generator=g, device=DEV) * (D * Hi) ** -0.5 - 0.1 * (D * Hi) ** -0.5
        if case["fmt"] == "bf16":
            s["q"], s["w"] = q.to(torch.bfloat16), w
        else:
            codes, sc = _pow2_quant(q)
            s["q"], s["w"] = codes.view(torch.uint8), (w * sc).contiguous()
        # columns past a row's visible blocks are not written
        s["scores"] = torch.full((T, -(-max(lens) // case["bt"])), NEG, device=DEV)
        return s
    if op == "select":
        W = -(-max(lens) // case["bt"])
        x = torch.randn((T, W), generator=g, device=DEV) * torch.rand((T, 1), generator=g, device=DEV).add_(0.1)
        s["scores"] = torch.round(x * case["grain"]) if case["grain"] else x
        s["num_blocks"] = nb
        return s
    H, k = case["H"], case["k"]
    q = torch.randn((T, H, 576), generator=g, device=DEV)
    if case["fmt"] == "bf16":
        s["kv"] = torch.randn((nb, ps, 576), generator=g, device=DEV).to(torch.bfloat16)
    elif case["fmt"] == "fp8":
        s["kv"] = (torch.randn((nb, ps, 576), generator=g, device=DEV) * 20).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        x = torch.randn((nb, ps, 4, 128), generator=g, device=DEV)
        codes, sc = _pow2_quant(x)
        s["kv"] = torch.cat([codes.view(torch.uint8).reshape(nb, ps, 512), sc.contiguous().view(torch.uint8).reshape(nb, ps, 16),
                             torch.randn((nb, ps, 64), generator=g, device=DEV).to(torch.bfloat16).view(torch.uint8)], -1).contiguous()
    s["q"] = (q * 20).to(torch.float8_e4m3fn).view(torch.uint8) if case["fmt"] == "fp8" else q.to(torch.bfloat16)
    s["qk"] = 0.05 if case["fmt"] == "fp8" else 1.0
    # the selected pages: the newest of every row and random others, ascending, -1 after them
    pages = torch.tensor([-(-v // ps) for v in _visible(case)], device=DEV).unsqueeze(1)
    col = torch.arange(int(pages.max()), device=DEV).unsqueeze(0)
    key = torch.rand((T, col.shape[1]), generator=g, device=DEV)
    key = torch.where(col == pages - 1, 2.0, torch.where(col < pages, key, -1.0))
    if key.shape[1] < k:
        key = torch.nn.functional.pad(key, (0, k - key.shape[1]), value=-1.0)
    val, idx = key.topk(k, dim=1)
    big = 1 << 30
    idx = torch.where(val < 0, big, idx).sort(1).values
    s["blocks"] = torch.where(idx == big, -1, idx).to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _rotate(x, cs):
    """The last 64 values rotated in pairs (2i, 2i + 1) in 32 bits, one product rounded before the sum."""
    if cs is None:
        return x
    while cs.dim() < x.dim():
        cs = cs.unsqueeze(-2)
    c, sn = cs[..., :32], cs[..., 32:]
    x0, x1 = x[..., NOPE::2], x[..., NOPE + 1::2]
    y0 = (x0.double() * c.double() - (x1 * sn).double()).float()
    y1 = (x1.double() * c.double() + (x0 * sn).double()).float()
    return torch.cat([x[..., :NOPE], torch.stack([y0, y1], -1).flatten(-2)], -1)


def _plain_insert(s):
    case = s["case"]
    cs = None if s["positions"] is None else s["cos_sin"][s["positions"]]
    q, k = _rotate(s["q"].float(), cs), _rotate(s["k"].float(), cs)
    w = s["w"] * s["weight_scale"]
    if case["fmt"] == "bf16":
        s["cache"].view(-1, D)[s["slots"]] = k.to(torch.bfloat16)
        return {"q": q.to(torch.bfloat16), "w": w, "cache": s["cache"]}
    qc, qs = _pow2_quant(q)
    kc, ks = _pow2_quant(k)
    s["cache"].view(-1, D)[s["slots"]] = kc.view(torch.uint8)
    s["scales"].view(-1)[s["slots"]] = ks
    return {"q": qc, "w": w * qs, "cache": s["cache"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def _values(cache, scales):
    if scales is None:
        return cache.float()
    return cache.view(torch.float8_e4m3fn).float() * scales.unsqueeze(-1)


def _row_request(cu, n):
    """Request of each of n rows, and the row's place in it."""
    row = torch.arange(n, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), row.to(torch.int32), right=True)
    return b, row - cu[b]


def _plain_gather(s):
    ps = s["case"]["ps"]
    b, i = _row_request(s["cu"], s["n"])
    blk = s["table"][b, i // ps].long()
    codes = s["cache"][blk, i % ps]
    return _values(codes, None if s["scales"] is None else s["scales"][blk, i % ps]).to(torch.bfloat16)


def _plain_scores(s):
    case = s["case"]
    ps, bt = case["ps"], case["bt"]
    T, Hi = s["w"].shape
    B = case["B"]
    b, i = _row_request(s["cu_q"], T)
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    W = s["scores"].shape[1]
    L = min(s["table"].shape[1] * ps, -(-W * bt // ps) * ps)
    tab = s["table"][:, :L // ps].long()
    keys = _values(s["cache"][tab], None if s["scales"] is None else s["scales"][tab]).reshape(B, L, D)
    m = int(max(_rows(case)))
    pick = (s["cu_q"][:-1].long().unsqueeze(1) + torch.arange(m, device=DEV)).clamp(max=T - 1)
    q = s["q"].float() if case["fmt"] == "bf16" else s["q"].view(torch.float8_e4m3fn).float()
    x = torch.matmul(q[pick].reshape(B, m * Hi, D), keys.transpose(1, 2)).relu_()
    x = torch.matmul(s["w"][pick].unsqueeze(2), x.view(B, m, Hi, L)).squeeze(2)        # [B, m, L]
    sc = x[b, i]
    vis = s["seq_lens"].long()[b] - n[b] + i + 1
    sc = sc.masked_fill(torch.arange(L, device=DEV) >= vis.unsqueeze(1), NEG)
    if bt > 1:
        pad = -L % bt
        sc = torch.nn.functional.pad(sc, (0, pad), value=NEG).view(T, -1, bt).amax(-1)
    return sc[:, :W].contiguous()


def _plain_select(s):
    case = s["case"]
    bt, k, ps = case["bt"], case["k"], case["ps"]
    T, W = s["scores"].shape
    b, i = _row_request(s["cu_q"], T)
    n = (s["cu_q"][1:] - s["cu_q"][:-1])
    vis = (s["seq_lens"][b] - n[b] + i + 1).long().unsqueeze(1)
    nblk = (vis + bt - 1) // bt
    col = torch.arange(W, device=DEV).unsqueeze(0)
    x = torch.where(torch.isnan(s["scores"]), NEG, s["scores"])
    x = torch.where((col < case["first"]) | (col >= nblk - case["last"]), float("inf"), x)
    x = torch.where(col < nblk, x, NEG)
    val, idx = x.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    if W < k:
        val, idx = torch.nn.functional.pad(val, (0, k - W), value=NEG), torch.nn.functional.pad(idx, (0, k - W))
    big = 1 << 30
    idx = torch.where(val == NEG, big, idx).sort(1).values
    blocks = torch.where(idx == big, -1, idx)
    out = {"blocks": blocks.to(torch.int32)}
    if case["slots"]:
        pos = blocks.unsqueeze(2) * bt + torch.arange(bt, device=DEV)
        have = (blocks.unsqueeze(2) >= 0) & (pos < vis.unsqueeze(2))
        page = s["table"][b.view(-1, 1, 1), (pos.clamp(min=0) // ps).clamp(max=s["table"].shape[1] - 1)]
        out["slots"] = torch.where(have, page * ps + pos % ps, -1).to(torch.int32).reshape(T, k * bt)
    return out


def _entries(kv, fmt, qk):
    if fmt == "bf16":
        return kv.float()
    if fmt == "fp8":
        return kv.view(torch.float8_e4m3fn).float() * qk
    sc = kv[..., 512:528].contiguous().view(torch.float32).repeat_interleave(128, -1)
    return torch.cat([kv[..., :512].contiguous().view(torch.float8_e4m3fn).float() * sc, kv[..., 528:].contiguous().view(torch.bfloat16).float()], -1)


def _plain_selected(s):
    case = s["case"]
    ps, k = case["ps"], case["k"]
    T, H, _ = s["q"].shape
    b, i = _row_request(s["cu_q"], T)
    n = s["cu_q"][1:] - s["cu_q"][:-1]
    vis = (s["seq_lens"][b] - n[b] + i + 1).view(-1, 1, 1)
    blk = s["blocks"].unsqueeze(2)
    have = ((blk >= 0) & (blk * ps + torch.arange(ps, device=DEV) < vis)).reshape(T, 1, k * ps)
    page = s["table"][b.unsqueeze(1), s["blocks"].clamp(min=0).long()].long()
    e = _entries(s["kv"][page], case["fmt"], s["qk"]).reshape(T, k * ps, 576)
    q = s["q"].view(torch.float8_e4m3fn).float() * s["qk"] if case["fmt"] == "fp8" else s["q"].float()
    x = torch.matmul(q, e.transpose(1, 2)) * 192 ** -0.5
    x = x.masked_fill(~have, NEG)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    return {"out": (torch.matmul(p, e[..., :512]) / l).to(torch.bfloat16), "lse": (m + torch.log(l)).squeeze(-1)}


# ------------------------------------------------------------------------------------------ one pass

def _own_run(s):
    import mla_latent_cache_attention_gb300 as mla
    case, op = s["case"], s["case"]["op"]
    if op == "insert":
        q, w = mla.index_q_cache_insert(s["q"], s["k"], s["w"], s["cache"], s["scales"], s["slots"], fmt=case["fmt"],
                                        weight_scale=s["weight_scale"], positions=s["positions"], cos_sin_cache=s["cos_sin"])
        if case["fmt"] == "bf16":
            return {"q": q, "w": w, "cache": s["cache"]}
        f8 = torch.float8_e4m3fn
        return {"q": q.view(f8), "w": w, "cache": s["cache"].view(f8), "scales": s["scales"]}
    if op == "gather":
        return mla.index_gather(s["cache"], s["scales"], s["table"], s["cu"], fmt=case["fmt"], num_tokens=s["n"])
    if op == "scores":
        return mla.index_scores(s["q"], s["w"], s["cache"], s["scales"], s["table"], s["seq_lens"], s["cu_q"], fmt=case["fmt"],
                                block_tokens=case["bt"], max_context=case["hi"], scores=s["scores"])
    if op == "select":
        blocks, slots = mla.index_select(s["scores"], s["seq_lens"], case["k"], s["cu_q"], block_tokens=case["bt"], first=case["first"],
                                         last=case["last"], block_table=s["table"] if case["slots"] else None, page_size=case["ps"],
                                         num_blocks=s["num_blocks"])
        return {"blocks": blocks, "slots": slots} if case["slots"] else {"blocks": blocks}
    out, lse = mla.selected_decode(s["q"], s["kv"], s["table"], s["seq_lens"], s["blocks"], s["cu_q"], fmt=case["fmt"],
                                   softmax_scale=192 ** -0.5, q_scale=s["qk"], k_scale=s["qk"], return_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own_run(state)
    return {"insert": _plain_insert, "gather": _plain_gather, "scores": _plain_scores, "select": _plain_select,
            "selected": _plain_selected}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ 64 bits

def _decode_e4m3(codes):
    """Values of E4M3 bytes from the format's definition."""
    c = torch.arange(256, device=DEV)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e.double() - 7))
    v = torch.where((c & 127) == 127, float("nan"), v)
    return torch.where(c >= 128, -v, v)[codes.view(torch.uint8).long()]


def exact(case, seed):
    s = prepare(case, seed)
    op, ps = case["op"], case["ps"]
    if op == "insert":
        T = case["B"]
        rot = {}
        for name in ("q", "k"):
            x = s[name].double().reshape(T, -1, D).clone()
            if case["rope"]:
                a = s["cos_sin"][s["positions"]].double()
                co, si = a[:, None, :32], a[:, None, 32:]
                u, v = x[..., NOPE::2].clone(), x[..., NOPE + 1::2].clone()
                x[..., NOPE::2], x[..., NOPE + 1::2] = u * co - v * si, v * co + u * si
            rot[name] = x
        w = s["w"].double() * s["weight_scale"]
        if case["fmt"] == "bf16":
            cache = s["cache"].double().reshape(-1, D)
            cache[s["slots"]] = rot["k"][:, 0]
            return {"q": rot["q"], "w": w, "cache": cache.reshape(s["cache"].shape)}
        # codes are whole steps of a format: only the weights and scales have a value in 64 bits
        k = {}
        for name, x in rot.items():
            top = x.abs().amax(-1)
            k[name] = torch.where(top == 0, torch.zeros_like(top), torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)))
        scales = s["scales"].double().reshape(-1)
        scales[s["slots"]] = 2.0 ** k["k"][:, 0]
        return {"q": None, "w": w * 2.0 ** k["q"], "cache": None, "scales": scales.reshape(s["scales"].shape)}
    table = s["table"].cpu()
    lens = _lens(case)

    def cached(bq):     # the cached index keys of one request, in order
        n = lens[bq]
        at = torch.tensor([int(table[bq, j // ps]) * ps + j % ps for j in range(0, n, ps)], device=DEV)
        at = (at.unsqueeze(1) + torch.arange(ps, device=DEV)).reshape(-1)[:n]
        if s["scales"] is None:
            return s["cache"].reshape(-1, D)[at].double()
        return _decode_e4m3(s["cache"].reshape(-1, D)[at]) * s["scales"].reshape(-1)[at].double()[:, None]

    if op == "gather":
        return torch.cat([cached(bq) for bq in range(case["B"])])
    rows = _rows(case)
    if op == "scores":
        q = s["q"].double() if case["fmt"] == "bf16" else _decode_e4m3(s["q"])
        bt, out, r = case["bt"], s["scores"].double(), 0
        for bq, nq in enumerate(rows):
            key = cached(bq).t().contiguous()
            step = max(1, (1 << 28) // (lens[bq] * case["Hi"]))
            for r0 in range(0, nq, step):
                r1 = min(nq, r0 + step)
                dot = (q[r + r0:r + r1].reshape(-1, D) @ key).clamp_(min=0).view(r1 - r0, case["Hi"], -1)
                v = torch.bmm(s["w"][r + r0:r + r1].double().unsqueeze(1), dot).squeeze(1)
                see = lens[bq] - nq + torch.arange(r0, r1, device=DEV)
                v[torch.arange(lens[bq], device=DEV) > see[:, None]] = NEG
                if bt > 1:
                    v = torch.cat([v, v.new_full((r1 - r0, -lens[bq] % bt), NEG)], 1).unflatten(1, (-1, bt)).amax(2)
                out[r + r0:r + r1, :v.shape[1]] = v
            r += nq
        return out
    if op == "select":
        return None         # whole numbers: the plain form's are the definition's
    vis, H = _visible(case), case["H"]
    if len(vis) * case["k"] * ps * H > 1 << 27:
        return None
    kv = s["kv"].reshape(-1, s["kv"].shape[-1])
    outs, lses = [], []
    r = 0
    for bq, nq in enumerate(rows):
        for _ in range(nq):
            pos = [j for c in s["blocks"][r].tolist() if c >= 0 for j in range(c * ps, min(vis[r], c * ps + ps))]
            at = torch.tensor([int(table[bq, j // ps]) * ps + j % ps for j in pos], device=DEV)
            x = kv[at]
            if case["fmt"] == "bf16":
                val = x.double()
            elif case["fmt"] == "fp8":
                val = _decode_e4m3(x) * s["qk"]
            else:
                sc = x[:, 512:528].contiguous().view(torch.float32).double()
                val = torch.cat([(_decode_e4m3(x[:, :512]).view(-1, 4, 128) * sc[:, :, None]).reshape(-1, 512),
                                 x[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
            qr = _decode_e4m3(s["q"][r]) * s["qk"] if case["fmt"] == "fp8" else s["q"][r].double()
            logit = qr @ val.t() * 192 ** -0.5
            lse = torch.logsumexp(logit, 1)
            outs.append(torch.exp(logit - lse[:, None]) @ val[:, :512])
            lses.append(lse)
            r += 1
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
