"""What is measured of the latent cache held in 4 bits and of the step around it: blocks and slots planned from
request lengths, rotary positions, the insert of new tokens into the 4-bit cache, its context read back, and the
paged decode over it.

Where ``own`` is false ``run`` computes the plain form with elementary torch operations; where it is true it
calls the framework.

A 4-bit record has 400 bytes: 512 E2M1 codes (value 2i in the low half of byte i), 16 bytes with the exponents of
the scales of its groups of 32 values (2^(byte - 127)), and 64 bf16 rope values.
"""
import math

import torch

own = False

DEV = "cuda"
NEG = float("-inf")
REC = 400
SCALE = 192 ** -0.5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a small batch: the queries concatenated and rotated, the latents written, and the new
        # entries read back
        dict(name="insert_decode", op="insert", way="decode", T=32, H=16, ps=64, rope=True),
        # a chunk of a long prefill, a ragged size: full keys, and the chunk's entries read back
        dict(name="insert_prefill", op="insert", way="prefill", T=8191, H=16, ps=64, rope=True),
        # the cached context of one short request read back
        dict(name="gather_short", op="gather", B=1, lo=1021, hi=1021, ps=64),
        # the cached context of a chunk of requests read back for a long prefill
        dict(name="gather_context", op="gather", B=13, lo=1024, hi=32768, ps=64),
        # one token of one short request: latency
        dict(name="decode_one", op="decode", B=1, q=1, H=16, lo=1021, hi=1021, ps=64),
        # a decode step of an ordinary batch
        dict(name="decode_batch", op="decode", B=32, q=1, H=16, lo=1024, hi=8192, ps=64),
        # four speculative tokens a request over long contexts
        dict(name="decode_verify", op="decode", B=64, q=4, H=16, lo=16384, hi=131072, ps=64),
        # a decode step of a large batch with many heads: bound by the products
        dict(name="decode_heads", op="decode", B=128, q=1, H=96, lo=8192, hi=32768, ps=64),
        # the rope part of the queries and the shared key of one decode step
        dict(name="rope_decode", op="rope", T=32, H=16, Hk=1, D=192, Dk=64, R=64, half=False, dtype="bf16", inverse=False),
        # a chunk of a long prefill, whole heads, in halves
        dict(name="rope_prefill", op="rope", T=8191, H=64, Hk=8, D=128, Dk=128, R=128, half=True, dtype="bf16", inverse=False),
        # the blocks and slots of one decode step of a large batch, some requests finished
        dict(name="plan_decode", op="plan", B=256, q=1, lo=1, hi=131072, ps=64, T=256),
        # the blocks and slots of a step that mixes prefill chunks
        dict(name="plan_prefill", op="plan", B=64, q=512, lo=0, hi=32768, ps=64, T=32768),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["insert", "gather", "decode", "decode", "decode", "rope", "rope", "plan"])
    ps = rng.choice([16, 32, 64, 128])
    if op == "insert":
        way = rng.choice(["decode", "prefill"])
        return dict(op=op, way=way, T=_spread(rng, 1, 512 if way == "decode" else 8192), H=rng.randint(1, 64 if way == "decode" else 16), ps=ps, rope=rng.random() < 0.8)
    if op == "gather":
        B = _spread(rng, 1, 32)
        hi = _spread(rng, 1, 200000 // B)
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, ps=ps)
    if op == "decode":
        q = rng.choice([1, 1, 1, 2, 4])
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 1, min(131072, 1500000 // (B * q)))
        return dict(op=op, B=B, q=q, H=rng.choice([16, 16, 32, 64, 96, 128, rng.randint(1, 128)]), lo=rng.randint(0, hi), hi=hi, ps=ps)
    if op == "rope":
        R = rng.choice([32, 64, 64, 128])
        H = rng.randint(1, 64)
        return dict(op=op, T=_spread(rng, 1, 8192), H=H, Hk=rng.choice([1, H, max(1, H // 8)]), D=R + rng.choice([0, 64, 128]), Dk=R + rng.choice([0, 0, 64]), R=R, half=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), inverse=rng.random() < 0.3)
    B, q = _spread(rng, 1, 512), rng.choice([1, 1, 4, _spread(rng, 1, 2048)])
    q = min(q, 32768 // B)
    hi = _spread(rng, 1, 4000000 // B)
    return dict(op=op, B=B, q=q, lo=rng.randint(0, hi), hi=hi, ps=ps, T=B * q + rng.choice([0, 0, 3, 64]))


# ------------------------------------------------------------------------------------------ shapes

def _lens(case):
    """Context lengths of the requests, spread over [lo, hi]; the last one is hi."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    return [hi if b == B - 1 else lo + int((hi - lo) * math.modf((b + 1) * 0.6180339887498949)[0]) for b in range(B)]


def _new(case):
    """Tokens of the step of every request: q, or in a step with prefill chunks ragged ones and single tokens."""
    q = case["q"]
    return [q if q < 16 or b == 0 else 1 if b % 3 == 1 else max(1, q - 37 * b % q) for b in range(case["B"])]


def _visible(case):
    """Visible tokens of every query row, rows grouped by request."""
    return [max(0, L - case["q"] + i + 1) for L in _lens(case) for i in range(case["q"])]


def work(case):
    op = case["op"]
    if op == "insert":
        T, H = case["T"], case["H"]
        # keys and queries of a prefill: [128 | 64] a head, the query's rotated part in place
        heads = H * 2 * 576 * 2 if case["way"] == "decode" else H * 2 * (128 + 192) + (H * 4 * 64 if case["rope"] else 0)
        entry = 2 * 576 + 8 + (264 if case["rope"] else 0) + REC
        back = T * (REC + 2 * 576)
        return {"bytes": T * (heads + entry) + back, "flops": T * (4 * 512 + (4 * 64 * (H + 1) if case["rope"] else 0))}
    if op == "gather":
        n = sum(_lens(case))
        return {"bytes": n * (REC + 2 * 576), "flops": n * 512}
    if op == "decode":
        vis, H = _visible(case), case["H"]
        return {"bytes": sum(_lens(case)) * REC + len(vis) * H * (576 * 2 + 512 * 2 + 4), "flops": sum(vis) * H * 2 * (576 + 512)}
    if op == "rope":
        n = case["T"] * (case["H"] * case["D"] + case["Hk"] * case["Dk"])
        return {"bytes": 2 * n * TYPES[case["dtype"]].itemsize + case["T"] * (8 + 4 * case["R"]), "flops": 3 * case["T"] * (case["H"] + case["Hk"]) * case["R"]}
    fin = sum(-(-L // case["ps"]) for b, L in enumerate(_lens(case)) if _finished(case, b))
    return {"bytes": 16 * case["T"] + 20 * case["B"] + 8 * fin + 8 * (sum(_new(case)) // case["ps"] + 1), "flops": case["T"]}


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


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


def _finished(case, b):
    """Every eighth request of a step is finished: its blocks go back, it has no tokens."""
    return b % 8 == 5


def _two(k):
    """2^k in 32 bits, k in [-126, 127]."""
    return ((k + 127).int() << 23).view(torch.float32)


def _quantised(x):
    """Codes [.., 256] and scale exponents [.., 16] of latents [.., 512]: the exponent of a group is the least k
    with amax <= 6 * 2^k, and no more than 14 below the record's largest; codes to the nearest, ties to even."""
    y = x.float().unflatten(-1, (16, 32))
    amax = y.abs().amax(-1)
    m, ex = torch.frexp(amax)
    k = torch.where(amax == 0, -1000, torch.where(m <= 0.75, ex - 3, ex - 2))
    k = torch.maximum(k, k.amax(-1, keepdim=True) - 14).clamp(min=-126)
    a = y.abs() * _two(-k).unsqueeze(-1)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).to(torch.uint8)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (k + 127).to(torch.uint8)


def _records(lat, rope):
    codes, ex = _quantised(lat)
    return torch.cat([codes, ex, rope.contiguous().view(torch.uint8)], -1)


def _cache(g, nb, ps):
    """Blocks of records of normalised latents, whose channels differ in size."""
    kv = torch.empty((nb, ps, REC), dtype=torch.uint8, device=DEV)
    chan = torch.exp(0.5 * torch.randn((512,), generator=g, device=DEV))
    step = max(1, (1 << 18) // ps)
    for i in range(0, nb, step):
        n = min(step, nb - i)
        lat = (torch.randn((n, ps, 512), generator=g, device=DEV) * chan).to(torch.bfloat16)
        kv[i:i + n] = _records(lat, torch.randn((n, ps, 64), generator=g, device=DEV).to(torch.bfloat16))
    return kv


def _angles(dim, n=131072):
    inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=DEV) / dim)
    ang = torch.arange(n, dtype=torch.float64, device=DEV).unsqueeze(1) * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case}
    rnd = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)      # noqa: E731
    if op == "insert":
        T, H, ps = case["T"], case["H"], case["ps"]
        if case["way"] == "decode":
            s["ql"], s["qpe"] = rnd(T, H, 512), rnd(T, H, 64)
        else:
            s["q"], s["kn"] = rnd(T, H, 192), rnd(T, H, 128)
        chan = torch.exp(0.5 * torch.randn((512,), generator=g, device=DEV))
        s["kv_c"], s["kpe"] = (rnd(T, 512).float() * chan).to(torch.bfloat16), rnd(T, 64)
        s["table"], nb = _table(g, [T], ps)
        s["slots"] = (s["table"][0].long().unsqueeze(1) * ps + torch.arange(ps, device=DEV)).reshape(-1)[:T].contiguous()
        s["cu"] = _i32([0, T])
        s["positions"] = s["cos_sin"] = None
        if case["rope"]:
            s["positions"], s["cos_sin"] = torch.randint(0, 131072, (T,), generator=g, device=DEV), _angles(64)
        s["cache"] = _cache(g, nb, ps)
        return s
    if op == "rope":
        T, dt = case["T"], TYPES[case["dtype"]]
        s["q"] = torch.randn((T, case["H"], case["D"]), generator=g, device=DEV).to(dt)
        s["k"] = torch.randn((T, case["Hk"], case["Dk"]), generator=g, device=DEV).to(dt)
        s["positions"], s["cos_sin"] = torch.randint(0, 131072, (T,), generator=g, device=DEV), _angles(case["R"])
        return s
    lens = _lens(case)
    ps = case["ps"]
    if op == "plan":
        B = case["B"]
        new = [0 if _finished(case, b) else n for b, n in enumerate(_new(case))]
        width = max(1, max(-(-(a + b) // ps) for a, b in zip(lens, new)))
        table, nb = _table(g, lens, ps, extra=0)
        s["table"] = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=0).contiguous()
        have = sum(new) // ps + B + 7
        freed = sum(-(-lens[b] // ps) for b in range(B) if _finished(case, b))
        s["free"] = torch.cat([nb + torch.randperm(have, generator=g, device=DEV).to(torch.int32), torch.zeros(freed, dtype=torch.int32, device=DEV)])
        s["num_free"] = _i32([have])
        s["seq"], s["new"] = _i32(lens), _i32(new)
        s["done"] = torch.tensor([_finished(case, b) for b in range(B)], device=DEV)
        return s
    s["table"], nb = _table(g, lens, ps)
    s["seq_lens"] = _i32(lens)
    s["cache"] = _cache(g, nb, ps)
    if op == "gather":
        s["cu"], s["n"] = _i32(_cum(lens)), sum(lens)
        return s
    s["q"] = rnd(case["B"] * case["q"], case["H"], 576)
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _values(rec):
    """Latents [.., 512] in 32 bits and rope values of records."""
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    b = torch.arange(256, device=DEV)
    pair = torch.stack([v[b & 15], v[b >> 4]], 1)
    lat = pair[rec[..., :256].int()].flatten(-2).unflatten(-1, (16, 32))
    sc = _two(rec[..., 256:272].int() - 127)
    return (lat * sc.unsqueeze(-1)).flatten(-2), rec[..., 272:].contiguous().view(torch.bfloat16)


def _turned(x, cs, at, half, inverse=False):
    """x [T, H, D] with the values at .. at + R rotated in 32 bits (cs [T, R]: cosines, then sines)."""
    n = cs.shape[1] // 2
    c, sn = cs[:, None, :n], cs[:, None, n:]
    if inverse:
        sn = -sn
    r = x[..., at:at + 2 * n].float()
    a, b = (r[..., :n], r[..., n:]) if half else (r[..., 0::2], r[..., 1::2])
    u, v = a * c - b * sn, b * c + a * sn
    y = torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([x[..., :at], y.to(x.dtype), x[..., at + 2 * n:]], -1)


def _read_back(s, n, cu):
    row = torch.arange(n, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), row.to(torch.int32), right=True)
    i = row - cu[b]
    ps = s["case"]["ps"]
    lat, rope = _values(s["cache"][s["table"][b, i // ps].long(), i % ps])
    return torch.cat([lat.to(torch.bfloat16), rope], -1)


def _plain_insert(s):
    case = s["case"]
    cs = s["cos_sin"][s["positions"]] if case["rope"] else None
    turn = lambda x: _turned(x, cs, x.shape[-1] - 64, False) if case["rope"] else x      # noqa: E731
    kpe = turn(s["kpe"].unsqueeze(1))
    if case["way"] == "decode":
        out = {"q": torch.cat([s["ql"], turn(s["qpe"])], -1)}
    else:
        out = {"q": turn(s["q"]), "k": torch.cat([s["kn"], kpe.expand(-1, case["H"], -1)], -1)}
    s["cache"].view(-1, REC)[s["slots"]] = _records(s["kv_c"], kpe.squeeze(1))
    return {**out, "entries": _read_back(s, case["T"], s["cu"])}


def _plain_decode(s):
    case = s["case"]
    B, q, H, ps = case["B"], case["q"], case["H"], case["ps"]
    L = s["table"].shape[1] * ps
    lat, rope = _values(s["cache"][s["table"].long()].view(B, L, REC))
    x = torch.matmul(s["q"][..., :512].float().view(B, q * H, 512), lat.transpose(1, 2))
    x += torch.matmul(s["q"][..., 512:].float().view(B, q * H, 64), rope.float().transpose(1, 2))
    x = x.mul_(SCALE).view(B, q, H, L)
    vis = s["seq_lens"].view(B, 1, 1, 1) - q + 1 + torch.arange(q, device=DEV).view(1, q, 1, 1)
    x = x.masked_fill_(torch.arange(L, device=DEV) >= vis, NEG)
    m = x.amax(-1, keepdim=True)
    p = torch.exp_(x.sub_(m.clamp(min=-1e38)))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, q * H, L), lat) / l.clamp(min=1e-38).view(B, q * H, 1)
    return {"out": o.view(B * q, H, 512).to(torch.bfloat16), "lse": (m + torch.log(l)).view(B * q, H)}


def _plain_rope(s):
    case = s["case"]
    cs = s["cos_sin"][s["positions"]]
    turn = lambda x: _turned(x, cs, x.shape[-1] - case["R"], case["half"], case["inverse"])      # noqa: E731
    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _plain_plan(s):
    case = s["case"]
    ps, T, B = case["ps"], case["T"], case["B"]
    seq, new, W = s["seq"].long(), s["new"].long(), s["table"].shape[1]
    # the blocks of finished requests go on top of the stack of free ones
    back = torch.where(s["done"], (seq + ps - 1) // ps, 0)
    end = back.cumsum(0)
    n = s["free"].shape[0]
    i = torch.arange(n, device=DEV) - s["num_free"]
    b = torch.searchsorted(end, i.clamp(min=0), right=True).clamp(max=B - 1)
    col = (i - (end - back)[b]).clamp(0, W - 1)
    s["free"].copy_(torch.where((i >= 0) & (i < end[-1]), s["table"][b, col], s["free"]))
    free = s["num_free"].long() + end[-1]
    # and every request takes what its new tokens need from the top
    seq = torch.where(s["done"], 0, seq)
    have, want = (seq + ps - 1) // ps, (seq + new + ps - 1) // ps
    need = want - have
    off = need.cumsum(0) - need
    c = torch.arange(W, device=DEV).unsqueeze(0)
    take = (c >= have.unsqueeze(1)) & (c < want.unsqueeze(1))
    at = (free - 1 - off.unsqueeze(1) - (c - have.unsqueeze(1))).clamp(0, n - 1)
    s["table"].copy_(torch.where(take, s["free"][at], s["table"]))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), new.cumsum(0)])
    row = torch.arange(T, device=DEV)
    rb = torch.searchsorted(cu[1:].contiguous(), row, right=True).clamp(max=B - 1)
    live = row < cu[-1]
    pos = torch.where(live, seq[rb] + row - cu[rb], 0)
    slot = torch.where(live, s["table"][rb, (pos // ps).clamp(max=W - 1)].long() * ps + pos % ps, -1)
    return {"slots": slot, "positions": pos, "cu": cu.int(), "seq": (seq + new).int(), "num_free": (free - need.sum()).int(), "table": s["table"], "free": s["free"]}


# ------------------------------------------------------------------------------------------ one pass

def _own_run(s):
    import mla_latent_cache_attention_gb300 as mla
    case, op = s["case"], s["case"]["op"]
    if op == "insert":
        if case["way"] == "decode":
            out = {"q": mla.q_concat_cache_insert(s["ql"], s["qpe"], s["kv_c"], s["kpe"], s["cache"], s["slots"], fmt="mxfp4", positions=s["positions"], cos_sin_cache=s["cos_sin"])}
        else:
            q = s["q"].clone()      # rotated in place
            k = mla.key_concat_cache_insert(q, s["kn"], s["kpe"], s["kv_c"], s["cache"], s["slots"], fmt="mxfp4", positions=s["positions"], cos_sin_cache=s["cos_sin"])
            out = {"q": q, "k": k}
        return {**out, "entries": mla.gather_context(s["cache"], s["table"], s["cu"], fmt="mxfp4", num_tokens=case["T"])}
    if op == "gather":
        return mla.gather_context(s["cache"], s["table"], s["cu"], fmt="mxfp4", num_tokens=s["n"])
    if op == "decode":
        out, lse = mla.paged_decode(s["q"], s["cache"], s["table"], s["seq_lens"], fmt="mxfp4", q_len=case["q"], max_context=max(1, case["hi"]), softmax_scale=SCALE, return_lse=True)
        return {"out": out, "lse": lse}
    if op == "rope":
        q, k = mla.rope(s["q"], s["positions"], s["cos_sin"], s["k"], layout="half" if case["half"] else "interleaved", inverse=case["inverse"])
        return {"q": q, "k": k}
    slots, positions, cu, seq, num_free = mla.plan_step(s["seq"], s["new"], s["table"], s["free"], s["num_free"], block_size=case["ps"], num_tokens=case["T"], finished=s["done"])
    return {"slots": slots, "positions": positions, "cu": cu, "seq": seq, "num_free": num_free, "table": s["table"], "free": s["free"]}


def run(state):
    if own:
        return _own_run(state)
    if state["case"]["op"] == "gather":
        return _read_back(state, state["n"], state["cu"])
    return {"insert": _plain_insert, "decode": _plain_decode, "rope": _plain_rope, "plan": _plain_plan}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ 64 bits

def _latents64(rec):
    """Latents and rope values of records [n, 400], from the formats' definitions."""
    b = rec[:, :256].long()
    c = torch.stack([b % 16, b // 16], 2).flatten(1)
    e, m = (c % 8) // 2, (c % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e.double() - 1)) * torch.where(c >= 8, -1.0, 1.0)
    sc = 2.0 ** (rec[:, 256:272].double() - 127)
    return v * sc.repeat_interleave(32, 1), rec[:, 272:].contiguous().view(torch.bfloat16).double()


def _rotated64(x, ang, first, pairs):
    """x with the values of `pairs` (index of the first and of the second of every pair) rotated."""
    y = x.double().clone()
    i, j = pairs
    co, si = ang[:, None, :i.numel()].double(), ang[:, None, i.numel():].double()
    y[..., first + i] = x[..., first + i].double() * co - x[..., first + j].double() * si
    y[..., first + j] = x[..., first + j].double() * co + x[..., first + i].double() * si
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None         # whole numbers: the plain form's are the definition's
    if op == "rope":
        R = case["R"]
        i = torch.arange(R // 2, device=DEV)
        pairs = (i, i + R // 2) if case["half"] else (2 * i, 2 * i + 1)
        ang = s["cos_sin"][s["positions"]].double()
        if case["inverse"]:
            ang[:, R // 2:] *= -1
        return {n: _rotated64(s[n], ang, s[n].shape[-1] - R, pairs) for n in ("q", "k")}
    ps = case["ps"]
    if op == "insert":
        T, H = case["T"], case["H"]
        i = torch.arange(32, device=DEV)
        ang = s["cos_sin"][s["positions"]] if case["rope"] else torch.cat([torch.ones((T, 32), device=DEV), torch.zeros((T, 32), device=DEV)], 1)
        turn = lambda x: _rotated64(x, ang, x.shape[-1] - 64, (2 * i, 2 * i + 1))      # noqa: E731
        kpe = turn(s["kpe"].view(T, 1, 64))
        if case["way"] == "decode":
            out = {"q": torch.cat([s["ql"].double(), turn(s["qpe"])], 2)}
        else:
            out = {"q": turn(s["q"]), "k": torch.cat([s["kn"].double(), kpe.expand(T, H, 64)], 2)}
        x = s["kv_c"].double().view(T, 16, 32)
        k = torch.ceil(torch.log2(x.abs().amax(2).clamp(min=1e-300) / 6))
        k = torch.maximum(k, k.amax(1, keepdim=True) - 14).clamp(min=-126)
        step = (2.0 ** k).unsqueeze(2)
        grid = torch.tensor([0, 1, 2, 4, 0.5, 1.5, 3, 6], dtype=torch.float64, device=DEV)     # even codes, then odd ones
        far = (x.abs() / step).unsqueeze(3) - grid
        near = (far.abs() + torch.tensor([0.0] * 4 + [1e-9] * 4, device=DEV)).argmin(3)
        lat = (grid[near] * torch.sign(x) * step).view(T, 512)
        return {**out, "entries": torch.cat([lat, kpe[:, 0]], 1)}
    table = s["table"].cpu()
    lens = _lens(case)
    flat = s["cache"].view(-1, REC)

    def cached(b):      # the records of one request, in order
        at = torch.tensor([int(table[b, j // ps]) * ps for j in range(0, lens[b], ps)], dtype=torch.int64, device=DEV)
        return flat[(at.unsqueeze(1) + torch.arange(ps, device=DEV)).reshape(-1)[:lens[b]]]

    if op == "gather":
        return torch.cat([torch.cat(_latents64(cached(b)), 1) for b in range(case["B"])])
    q, outs, lses = case["q"], [], []
    for b in range(case["B"]):
        lat, rope = _latents64(cached(b))
        for i in range(q):
            n = max(0, lens[b] - q + i + 1)
            x = s["q"][b * q + i].double()
            logit = (x[:, :512] @ lat[:n].t() + x[:, 512:] @ rope[:n].t()) * SCALE
            lse = torch.logsumexp(logit, 1) if n else torch.full((case["H"],), NEG, dtype=torch.float64, device=DEV)
            outs.append(torch.exp(logit - lse.unsqueeze(1)) @ lat[:n] if n else torch.zeros((case["H"], 512), dtype=torch.float64, device=DEV))
            lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
