"""The serving operators around the Engram forward, as measured: the cases, their inputs, one pass
of each in plain torch (``own`` false) or through the package (``own`` true), the bytes and
operations a pass cannot do without, and the results in 64 bits.

* ``residual_norm``: closes a block (norm of its output, gate, residual scale) and opens the next.
* ``linear``: matrix product with bias, activation (plain or gated) and residual.
* ``batch_plan``: block tables and slot maps of a ragged batch from its requests' lengths.
* ``hash_ids_paged``: the hash step of such a batch, its history in the plan's pages.
"""
import math

import torch

own = False

DEV = "cuda"
PAD_ID = 2            # the model's hash step: 2 layers, 4-grams, 8 heads, 99,092 compressed ids
LAYERS, NGRAM, HEADS = 2, 4, 8
VOCAB, COMPRESSED = 129_280, 99_092
COLS = (NGRAM - 1) * HEADS


def listed():
    return [
        # the residual seam behind the Engram block while 64 sequences decode: the value is the
        # last fifth of each token's projection row, the gate one number per token and stream
        dict(name="seam_decode_64", op="residual_norm", M=64, hc=4, dim=5120, ys=1, fp32=False, gate="token", post=True, strided=True),
        # the same seam over a prompt of 8192 tokens
        dict(name="seam_prefill_8192", op="residual_norm", M=8192, hc=4, dim=5120, ys=1, fp32=False, gate="token", post=True, strided=True),
        # a one-stream block with a fp32 residual stream and a gate per feature, an odd chunk
        dict(name="block_fp32_997", op="residual_norm", M=997, hc=1, dim=4096, ys=1, fp32=True, gate="feature", post=True, strided=False),
        # one token through a square projection added to the stream: latency
        dict(name="linear_token", op="linear", M=1, K=5120, N=5120, act="none", glu=False, bias=False, residual=True, fp32=False),
        # the value and key projection of 64 decoding sequences, with a bias
        dict(name="linear_decode_64", op="linear", M=64, K=6144, N=25600, act="none", glu=False, bias=True, residual=False, fp32=False),
        # the gated half of a feed-forward block over a ragged chunk
        dict(name="linear_glu_301", op="linear", M=301, K=5120, N=10240, act="silu", glu=True, bias=False, residual=False, fp32=False),
        # its second half, added to a fp32 residual stream
        dict(name="linear_down_1000", op="linear", M=1000, K=10240, N=5120, act="none", glu=False, bias=True, residual=True, fp32=True),
        # a prompt of 8192 tokens through the large projection with an activation
        dict(name="linear_prefill_8192", op="linear", M=8192, K=6144, N=25600, act="gelu", glu=False, bias=True, residual=False, fp32=False),
        # a decode step of 64 requests: one new token each
        dict(name="plan_decode_64", op="batch_plan", R=64, tokens=64, block=16, max_ctx=4096),
        # a full step of many requests: chunks of prompts, decoding and finished requests
        dict(name="plan_mixed_16384", op="batch_plan", R=512, tokens=16384, block=16, max_ctx=8192),
        # row ids of both Engram layers for 64 decoding requests
        dict(name="hash_decode_64", op="hash_ids_paged", R=64, tokens=64, block=16, max_ctx=4096),
        # row ids of a step of 8192 tokens over ragged requests
        dict(name="hash_mixed_8192", op="hash_ids_paged", R=96, tokens=8192, block=64, max_ctx=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["residual_norm", "linear", "linear", "batch_plan", "hash_ids_paged"])
    if op == "residual_norm":
        hc = rng.choice([1, 2, 4])
        return dict(op=op, M=_log(rng, 1, 8192), hc=hc, dim=8 * _log(rng, 16, 1024 if hc < 4 else 640), ys=rng.choice([1, hc]),
                    fp32=rng.random() < 0.3, gate=rng.choice(["none", "token", "feature"]), post=rng.random() < 0.7,
                    strided=rng.random() < 0.5)
    if op == "linear":
        glu = rng.random() < 0.3
        return dict(op=op, M=_log(rng, 1, 8192), K=8 * _log(rng, 16, 768), N=_log(rng, 64, 12800 if glu else 25600),
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]), glu=glu, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, fp32=rng.random() < 0.3)
    if op == "batch_plan":
        R = _log(rng, 1, 1024)
        return dict(op=op, R=R, tokens=max(R, _log(rng, 16, 16384)), block=rng.choice([1, 16, 24, 64, 256]), max_ctx=_log(rng, 300, 8192))
    R = _log(rng, 1, 256)
    return dict(op=op, R=R, tokens=max(R, _log(rng, 16, 8192)), block=rng.choice([16, 24, 64, 256]), max_ctx=_log(rng, 300, 8192))


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def _uniform(g, *shape):
    return torch.rand(shape, device=DEV, generator=g)


def _norm_inputs(c, g):
    M, hc, dim, ys = c["M"], c["hc"], c["dim"], c["ys"]
    x = _normal(g, 1, M, hc, dim, dtype=torch.float32)
    x *= torch.where(_uniform(g, 1, M, 1, 1) < 0.02, 50.0, 1.0)  # outlier tokens
    s = dict(c, x=x if c["fp32"] else x.bfloat16())
    if c["strided"]:  # the last ys * dim features of a wider projection row
        s["y"] = _normal(g, 1, M, (ys + 4) * dim)[..., 4 * dim:].view(1, M, ys, dim)
    else:
        s["y"] = _normal(g, 1, M, ys, dim)
    s["gate_in"] = None
    if c["gate"] == "token":
        s["gate_in"] = _uniform(g, 1, M, hc)
    elif c["gate"] == "feature":
        s["gate_in"] = _normal(g, 1, M, ys, dim, std=2.0)
    s["post_weight"] = _normal(g, hc, dim, std=0.1, dtype=torch.float32) + 1.0
    s["pre_weight"] = _normal(g, hc, dim, std=0.1, dtype=torch.float32) + 1.0
    s["mask"] = (_uniform(g, 1, M) >= 0.05).to(torch.uint8)
    s["alpha"], s["beta"], s["eps"] = 1.0, 0.75, 1e-6
    return s


def _linear_inputs(c, g):
    M, K, N = c["M"], c["K"], c["N"]
    rows = 2 * N if c["glu"] else N
    s = dict(c, x=_normal(g, M, K), w=_normal(g, rows, K, std=K ** -0.5))
    s["bias_in"] = _normal(g, rows, std=0.5, dtype=torch.float32) if c["bias"] else None
    s["res"] = _normal(g, M, N, dtype=torch.float32 if c["fp32"] else torch.bfloat16) if c["residual"] else None
    return s


def _plan_inputs(c, g):
    """Requests with pages in a shuffled pool: most decode (one new token), some bring a part of a
    prompt (in all about the step's tokens), some are idle or finished."""
    R, bs, tokens = c["R"], c["block"], c["tokens"]
    max_blocks = -(-c["max_ctx"] // bs) + 1
    cap = max_blocks * bs
    held = (_uniform(g, R) * c["max_ctx"] * 0.7).long()
    kind = _uniform(g, R)
    share = max(1, 4 * (tokens - R) // R)
    new = torch.where(kind < 0.5, 1 + (_uniform(g, R) * min(share, cap)).long(), 1)
    if R == tokens:
        new = torch.ones_like(new)
    new = torch.where(kind > 0.96, 0, new)
    new = torch.where(kind > 0.98, -1, new)
    if R == 1:
        new = new.clamp(1, tokens)
    held = torch.where(held + new > cap, cap - torch.clamp(new, 0), held)
    n_pages = R * max_blocks
    order = torch.argsort(_uniform(g, n_pages)).to(torch.int32)
    table = order.view(R, max_blocks).clone()
    have = (held + bs - 1) // bs
    spare = torch.arange(max_blocks, device=DEV)[None] >= have[:, None]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    free[: int(spare.sum())] = table[spare]
    table[spare] = -1
    s = dict(c, max_blocks=max_blocks, n_blocks=n_pages)
    s |= dict(new_lens=new.to(torch.int32), cached_lens=held.to(torch.int32), block_table=table, free_list=free,
              free_count=spare.sum().to(torch.int32).reshape(1))
    return s


def _primes():
    """24 primes above 16,000,000 for each layer, as the model's tables have."""
    found, n = [], 16_000_001
    while len(found) < LAYERS * COLS:
        if all(n % d for d in range(3, int(n ** 0.5) + 1, 2)):
            found.append(n)
        n += 2
    return found


_PRIMES = []


def _hash_inputs(c, g):
    """Tokens of a planned step: the plan of the requests above, their token ids and the history."""
    s = _plan_inputs(c, g)
    if not _PRIMES:
        _PRIMES.extend(_primes())
    primes = torch.tensor(_PRIMES, dtype=torch.int64, device=DEV).view(LAYERS, NGRAM - 1, HEADS)
    flat = primes.view(LAYERS, COLS)
    s["primes"] = primes
    s["offsets"] = torch.cumsum(flat, 1) - flat
    s["token_map"] = torch.randint(0, COMPRESSED, (VOCAB,), generator=g, device=DEV, dtype=torch.int32)
    s["multipliers"] = torch.randint(-2 ** 62, 2 ** 62, (LAYERS, NGRAM), generator=g, device=DEV, dtype=torch.int64) * 2 + 1
    s["ids"] = torch.randint(0, VOCAB, (c["tokens"],), generator=g, device=DEV, dtype=torch.int64)
    s["mask"] = (_uniform(g, c["tokens"]) >= 0.03).to(torch.uint8)  # image spans take no part
    s["history"] = torch.randint(0, COMPRESSED, (s["n_blocks"], c["block"]), generator=g, device=DEV, dtype=torch.int64)
    s["plan"] = _plain_plan(s)  # what the step's plan says, in hand before its hash
    return s


def prepare(case, seed):
    g = _gen(seed)
    return {"residual_norm": _norm_inputs, "linear": _linear_inputs, "batch_plan": _plan_inputs, "hash_ids_paged": _hash_inputs}[case["op"]](case, g)


# ---------------------------------------------------------------- plain forms


def _plain_norm(s):
    x, y = s["x"].float(), s["y"].float()
    n = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) if s["post"] else y
    n = n * s["post_weight"]
    if s["gate"] == "token":
        n = n * s["gate_in"].unsqueeze(-1)
    elif s["gate"] == "feature":
        n = n / (1.0 + torch.exp(-s["gate_in"].float()))
    r = torch.where(s["mask"].bool()[..., None, None], s["alpha"] * x + s["beta"] * n, x)
    h = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + s["eps"]) * s["pre_weight"]
    return {"out": r.to(s["x"].dtype), "h": h.bfloat16()}


def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z * 0.5 * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    return z


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias_in"] is not None:
        z = z + s["bias_in"]
    if s["glu"]:
        z = _plain_act(z[:, : s["N"]], s["act"]) * z[:, s["N"]:]
    else:
        z = _plain_act(z, s["act"])
    if s["res"] is not None:
        z = z + s["res"].float()
    return z.to(torch.float32 if s["fp32"] else torch.bfloat16)


def _plain_plan(s):
    R, bs, mb, nb, T = s["R"], s["block"], s["max_blocks"], s["n_blocks"], s["tokens"]
    new, held = s["new_lens"].long(), s["cached_lens"].long()
    table, free = s["block_table"].view(-1), s["free_list"]
    bad = (held < 0) | (held > mb * bs) | ((new > 0) & (held + new > mb * bs))
    gone = (new < 0) & ~bad
    have = torch.where(bad, 0, (held + bs - 1) // bs)
    # finished requests' blocks on top of the stack
    back = torch.where(gone, have, 0)
    free0 = s["free_count"].long().clamp(0, nb)
    cols = torch.arange(mb, device=DEV)[None]
    at = free0 + (torch.cumsum(back, 0) - back)[:, None] + cols
    at = torch.where((cols < back[:, None]) & (at < nb), at, nb)
    pool = torch.cat([free, free.new_zeros(1)])
    pool[at.view(-1)] = table
    free.copy_(pool[:nb])
    avail = (free0 + back.sum()).clamp(max=nb)
    # admitted in order: by tokens, then by blocks
    want = torch.where(bad | (new < 0), 0, new)
    status = torch.where(bad, 3, 0)
    over = (want > 0) & (torch.cumsum(want, 0) > T)
    status = torch.where(over, 1, status)
    want = torch.where(over, 0, want)
    need = torch.where(want > 0, (held + want + bs - 1) // bs - have, 0)
    short = (need > 0) & (torch.cumsum(need, 0) > avail)
    status = torch.where(short, 2, status)
    want = torch.where(short, 0, want)
    need = torch.where(short, 0, need)
    tok_end, blk_end = torch.cumsum(want, 0), torch.cumsum(need, 0)
    # new entries of the tables, from the top of the stack down
    e = torch.arange(T, device=DEV)
    r = torch.searchsorted(blk_end, e, right=True).clamp(max=R - 1)
    to = r * mb + have[r] + e - (blk_end - need)[r]
    grown = torch.cat([table, table.new_zeros(1)])
    grown[torch.where(e < blk_end[-1], to, R * mb)] = free[(avail - 1 - e).clamp(min=0)]
    table.copy_(grown[: R * mb])
    # tokens
    live = e < tok_end[-1]
    r = torch.searchsorted(tok_end, e, right=True).clamp(max=R - 1)
    pos = held[r] + e - (tok_end - want)[r]
    page = table[r * mb + torch.where(live, pos // bs, 0)].long()
    slots = torch.where(live & (page >= 0) & (page < nb), page * bs + pos % bs, -1)
    return dict(token_start=torch.cat([tok_end.new_zeros(1), tok_end]).to(torch.int32), start_pos=s["cached_lens"].clone(),
                seq_lens=torch.where(gone, 0, held + want).to(torch.int32), status=status.to(torch.int32),
                free_left=(avail - blk_end[-1]).to(torch.int32).reshape(1), slots=slots,
                positions=torch.where(live, pos, -1).to(torch.int32), requests=torch.where(live, r, -1).to(torch.int32),
                live=live.to(torch.uint8))


def _plain_hash(s):
    p, bs, nb = s["plan"], s["block"], s["n_blocks"]
    T = s["tokens"]
    ids = s["ids"]
    known = (ids >= 0) & (ids < VOCAB) & s["mask"].bool()
    comp = torch.where(known, s["token_map"].long()[ids.clamp(0, VOCAB - 1)], -1)
    req, pos = p["requests"].long(), p["positions"].long()
    live = req >= 0
    r = req.clamp(min=0)
    first = p["start_pos"].long()[r]
    hist = s["history"].view(-1)
    i = torch.arange(T, device=DEV)
    blocked = ~live
    toks = []
    for shift in range(NGRAM):
        q = pos - shift
        page = s["block_table"][r, (q.clamp(min=0) // bs)].long()
        old = hist[(page * bs + q.clamp(min=0) % bs).clamp(0, nb * bs - 1)]
        old = torch.where((page >= 0) & (page < nb), old, -1)
        src = torch.where(q >= first, comp[(i - shift).clamp(min=0)], old)
        blocked = blocked | (q < 0) | (src == -1)
        toks.append(torch.where(blocked, PAD_ID, src))
    m = s["multipliers"]
    rolling = toks[0] * m[:, :1]
    out = torch.empty((LAYERS, T, NGRAM - 1, HEADS), dtype=torch.int64, device=DEV)
    for n in range(1, NGRAM):
        rolling = rolling ^ (toks[n] * m[:, n:n + 1])
        out[:, :, n - 1] = torch.remainder(rolling[:, :, None], s["primes"][:, None, n - 1])
    grown = torch.cat([hist, hist.new_zeros(1)])
    grown[torch.where(p["slots"] >= 0, p["slots"], nb * bs)] = comp
    hist.copy_(grown[: nb * bs])
    return {"hash_ids": out.view(LAYERS, T, COLS) + s["offsets"][:, None], "history": s["history"]}


def _plain(s):
    if s["op"] == "residual_norm":
        return _plain_norm(s)
    if s["op"] == "linear":
        return _plain_linear(s)
    if s["op"] == "batch_plan":
        return dict(_plain_plan(s), block_table=s["block_table"], free_list=s["free_list"])
    return _plain_hash(s)


# ---------------------------------------------------------------- the package's calls


def _handle(s):
    """What a program keeps beside its tensors: the layout, and for a plan its buffers."""
    import hashed_gram_engram_amd as eg
    if s["op"] == "residual_norm":
        gate = {"none": eg.GATE_NONE, "token": eg.GATE_TOKEN, "feature": eg.GATE_FEATURE}[s["gate"]]
        return eg, eg.make_norm_layout(s["hc"], s["dim"], y_streams=s["ys"], gate=gate, post_norm=s["post"], alpha=s["alpha"],
                                       beta=s["beta"], post_eps=s["eps"], pre_eps=s["eps"],
                                       stream_format=eg.STREAM_FP32 if s["fp32"] else eg.STREAM_BF16)
    if s["op"] == "linear":
        act = {"none": eg.ACT_NONE, "relu": eg.ACT_RELU, "gelu": eg.ACT_GELU, "gelu_tanh": eg.ACT_GELU_TANH, "silu": eg.ACT_SILU,
               "sigmoid": eg.ACT_SIGMOID}[s["act"]]
        return eg, eg.make_linear_layout(s["K"], s["N"], activation=act, glu=s["glu"],
                                         stream_format=eg.STREAM_FP32 if s["fp32"] else eg.STREAM_BF16)
    pages = eg.make_page_layout(s["block"], s["max_blocks"], s["n_blocks"])
    if s["op"] == "batch_plan":
        return eg, pages, eg.BatchPlan(s["R"], s["tokens"], device=DEV)
    plan = eg.BatchPlan(s["R"], s["tokens"], device=DEV)
    for name, t in s["plan"].items():
        getattr(plan, name).copy_(t)
    return eg, pages, plan, eg.make_hash_layout(LAYERS, NGRAM, HEADS, PAD_ID, VOCAB, s["max_blocks"] * s["block"])


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    eg, lay = s["handle"][:2]
    if s["op"] == "residual_norm":
        out, h = eg.engram_residual_norm(lay, s["x"], s["y"], gate=s["gate_in"], post_weight=s["post_weight"],
                                         pre_weight=s["pre_weight"], token_mask=s["mask"])
        return {"out": out, "h": h}
    if s["op"] == "linear":
        return eg.engram_linear(lay, s["x"], s["w"], bias=s["bias_in"], residual=s["res"])
    plan = s["handle"][2]
    if s["op"] == "batch_plan":
        eg.engram_batch_plan(lay, s["new_lens"], s["cached_lens"], s["block_table"], s["free_list"], s["free_count"], plan)
        return dict({k: getattr(plan, k) for k in eg.BatchPlan.FIELDS}, block_table=s["block_table"], free_list=s["free_list"])
    ids = eg.engram_hash_ids_paged(s["handle"][3], lay, s["token_map"], s["multipliers"], s["primes"], s["offsets"], s["ids"], plan,
                                   s["block_table"], s["history"], token_mask=s["mask"])
    return {"hash_ids": ids, "history": s["history"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- floors and exact results


def work(case):
    c = case
    if c["op"] == "residual_norm":
        e = c["M"] * c["hc"] * c["dim"]
        shared = c["M"] * c["ys"] * c["dim"]
        n = e * (4 if c["fp32"] else 2) * 2 + e * 2 + shared * 2 + 8 * c["hc"] * c["dim"] + c["M"]
        n += {"none": 0, "token": 4 * c["M"] * c["hc"], "feature": 2 * shared}[c["gate"]]
        return {"bytes": n, "flops": 10 * e}
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        rows = 2 * N if c["glu"] else N
        o = 4 if c["fp32"] else 2
        return {"bytes": 2 * (M * K + rows * K) + 4 * rows * c["bias"] + M * N * o * (1 + c["residual"]), "flops": 2 * M * rows * K}
    if c["op"] == "batch_plan":
        # lengths, new pages (popped and written), slots, positions, requests and marks
        return {"bytes": 24 * c["R"] + 8 * (c["tokens"] // c["block"]) + 17 * c["tokens"], "flops": 0}
    # ids, masks, map, positions, slots and requests read; row ids and history written
    return {"bytes": c["tokens"] * (8 + 1 + 4 + 8 + 4 + 4 + 8 + 8 * LAYERS * COLS), "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "linear":
        w, x = s["w"].double(), s["x"].double()
        z = torch.mm(x, w.transpose(0, 1).contiguous())
        del w, x
        if s["bias_in"] is not None:
            z += s["bias_in"].double()
        a = z[:, : s["N"]] if s["glu"] else z
        f = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "sigmoid": lambda v: (1 + (-v).exp()).reciprocal(),
             "silu": lambda v: v * (1 + (-v).exp()).reciprocal(), "gelu": lambda v: 0.5 * v * (1 + torch.erf(v / 2 ** 0.5)),
             "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3)))}[s["act"]]
        a = f(a)
        if s["glu"]:
            a = a * z[:, s["N"]:]
        return a + s["res"].double() if s["res"] is not None else a
    if s["op"] != "residual_norm":
        return None  # whole numbers
    outs, hs = [], []
    for m0 in range(0, s["M"], 1024):  # some tokens at a time
        x, y = s["x"][0, m0:m0 + 1024].double(), s["y"][0, m0:m0 + 1024].double()
        if s["post"]:
            y = y / ((y * y).sum(-1, keepdim=True) / s["dim"] + s["eps"]).sqrt()
        y = y * s["post_weight"].double()
        if s["gate"] != "none":
            k = s["gate_in"][0, m0:m0 + 1024].double()
            y = y * (k[..., None] if s["gate"] == "token" else (1 + (-k).exp()).reciprocal())
        opened = s["mask"][0, m0:m0 + 1024].double()[:, None, None]
        # a closed token keeps its stream as it is
        r = torch.where(opened > 0, x * s["alpha"] + y * s["beta"], x)
        outs.append(r)
        hs.append(r / ((r * r).sum(-1, keepdim=True) / s["dim"] + s["eps"]).sqrt() * s["pre_weight"].double())
    return {"out": torch.cat(outs)[None], "h": torch.cat(hs)[None]}
