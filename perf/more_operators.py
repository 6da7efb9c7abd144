"""The latent cache and the attention that reads it, as measured: the cases, their inputs, one pass of each
in plain torch (``own`` false) or through the package (``own`` true), the bytes and operations a pass
cannot do without, and the results in 64 bits.

* ``cache``: a step's latent rows into the plan's pages (bf16, or e4m3 codes with a power-of-two scale for
  each 32 features), then the rows of the step's requests back as bf16.
* ``absorbed``: attention of queries in the latent space over the paged rows, for decoding.
* ``expanded``: attention over per-head keys and values made from the rows, for prompts.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the next turn of a few short conversations, odd lengths
        dict(name="cache_turns_6", op="cache", R=6, new=23, even=False, ctx=700, block=16, dc=512, dr=64, fp8=True),
        # prompts of two dozen requests behind what they hold already
        dict(name="cache_prompts_24", op="cache", R=24, new=1024, even=False, ctx=8192, block=64, dc=512, dr=64, fp8=True),
        # the same kept in bf16, a smaller latent, pages that no tile fits
        dict(name="cache_bf16_10", op="cache", R=10, new=900, even=False, ctx=5000, block=24, dc=256, dr=32, fp8=False),
        # a decode step of three short requests: latency
        dict(name="decode_short_3", op="absorbed", R=3, new=1, even=True, ctx=90, block=16, H=8, dc=128, dr=32, hd=64, fp8=False, window=0),
        # one request decoding behind a long document
        dict(name="decode_long_1", op="absorbed", R=1, new=1, even=True, ctx=65536, block=64, H=128, dc=512, dr=64, hd=128, fp8=True, window=0),
        # 64 decoding requests of ragged lengths, every head on this device
        dict(name="decode_64", op="absorbed", R=64, new=1, even=True, ctx=8192, block=64, H=128, dc=512, dr=64, hd=128, fp8=True, window=0),
        # 128 decoding requests with an eighth of the heads, the cache in bf16
        dict(name="decode_bf16_128", op="absorbed", R=128, new=1, even=True, ctx=8192, block=16, H=16, dc=512, dr=64, hd=128, fp8=False, window=0),
        # drafts of five tokens being verified, a sliding window, odd pages
        dict(name="draft_32", op="absorbed", R=32, new=5, even=True, ctx=3001, block=24, H=32, dc=256, dr=64, hd=128, fp8=True, window=2000),
        # one short prompt: latency
        dict(name="prompt_37", op="expanded", R=1, new=37, even=True, ctx=37, H=16, dr=32, hd=64, window=0),
        # ragged parts of prompts, a sliding window, an odd number of heads
        dict(name="prompts_12", op="expanded", R=12, new=1500, even=False, ctx=3500, H=20, dr=64, hd=128, window=1000),
        # a short part of a prompt behind a long document
        dict(name="chunk_512", op="expanded", R=1, new=512, even=True, ctx=16896, H=16, dr=64, hd=128, window=0),
        # a prompt of 8192 tokens
        dict(name="prompt_8192", op="expanded", R=1, new=8192, even=True, ctx=8192, H=64, dr=64, hd=128, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "absorbed", "absorbed", "expanded", "expanded"])
    if op == "cache":
        R, new = _log(rng, 1, 64), _log(rng, 1, 1024)
        ctx = new + _log(rng, 1, max(2, min(8192, 190_000 // R) - new))
        return dict(op=op, R=R, new=new, even=rng.random() < 0.3, ctx=ctx, block=rng.choice([1, 16, 24, 64, 256]),
                    dc=rng.choice([128, 256, 512, 512]), dr=rng.choice([32, 64, 64]), fp8=rng.random() < 0.6)
    if op == "absorbed":
        while True:
            R, new, H, ctx = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 5, 11]), rng.choice([1, 4, 16, 20, 32, 64, 96, 128]), _log(rng, 40, 65536)
            if R * ctx <= 128 * 8192 and R * ctx * H * new <= 48 * 8192 * 128:
                break
        return dict(op=op, R=R, new=new, even=rng.random() < 0.8, ctx=ctx, block=rng.choice([1, 16, 24, 64, 256]), H=H,
                    dc=rng.choice([128, 256, 512, 512, 512]), dr=rng.choice([32, 64, 64]), hd=rng.choice([64, 128]),
                    fp8=rng.random() < 0.5, window=rng.choice([0, 0, 0, _log(rng, 1, ctx)]))
    while True:
        R, new, H = _log(rng, 1, 16), _log(rng, 1, 8192), rng.choice([1, 4, 16, 20, 32, 64])
        ctx = new + rng.choice([0, _log(rng, 1, 16384)])
        if R * new * ctx * H <= 8192 * 8192 * 32 and R * ctx * H <= 1_000_000:
            break
    return dict(op=op, R=R, new=new, even=rng.random() < 0.5, ctx=ctx, H=H, dr=rng.choice([32, 64, 64]),
                hd=rng.choice([64, 128, 128]), window=rng.choice([0, 0, 0, _log(rng, 1, ctx)]))


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def _lens(c):
    """New and cached tokens of each request on the host: what a case computes does not depend on the
    seed.  One request in 24 is idle."""
    R, new, ctx = c["R"], c["new"], c["ctx"]
    g = torch.Generator().manual_seed(R * 1_000_003 + new * 1009 + ctx)
    u, v = torch.rand(R, generator=g), torch.rand(R, generator=g)
    n = torch.full((R,), new) if c["even"] else 1 + (u * new).long().clamp(max=new - 1)
    held = ((ctx - n) * (1.0 if R == 1 else 0.4 + 0.6 * v)).long()
    n[23::24] = 0
    return n, held


def _plan_inputs(c, g):
    """The step's plan, in hand: pages in a shuffled pool, some room behind the last token."""
    new, held = (t.to(DEV) for t in _lens(c))
    live = int(new.sum())
    T = live if c["R"] == 1 else live + live // 16 + 1
    start = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    e = torch.arange(T, device=DEV)
    r = torch.searchsorted(start[1:], e, right=True).clamp(max=c["R"] - 1)
    used = e < live
    pos = held[r] + e - start[r]
    i32 = torch.int32
    s = dict(c, T=T)
    p = dict(token_start=start.to(i32), start_pos=held.to(i32), seq_lens=(held + new).to(i32), status=torch.zeros_like(new).to(i32),
             free_left=torch.zeros(1, dtype=i32, device=DEV), positions=torch.where(used, pos, -1).to(i32),
             requests=torch.where(used, r, -1).to(i32), live=used.to(torch.uint8))
    p["slots"] = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    if "block" in c:
        bs = c["block"]
        mb = -(-c["ctx"] // bs)
        table = torch.argsort(torch.rand(c["R"] * mb, device=DEV, generator=g)).to(i32).view(c["R"], mb)
        page = table[r, (pos // bs).clamp(0, mb - 1)].long()
        p["slots"] = torch.where(used, page * bs + pos % bs, -1)
        s |= dict(table=table, max_blocks=mb, n_blocks=c["R"] * mb)
    s["plan"] = p
    return s


def _pool(s, g):
    """A pool whose every row holds a latent: the requests' own, and what others left."""
    n = s["n_blocks"] * s["block"]
    rows = _rows(s, _normal(g, n, s["dc"]), _normal(g, n, s["dr"]))
    return rows.view(s["n_blocks"], s["block"], -1)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = _plan_inputs(c, g)
    T = s["T"]
    if c["op"] == "cache":
        new, held = _lens(c)
        rows = int((new + held)[new > 0].sum())
        s["pool"] = _pool(s, g)
        # the projection's rows: the latent, then the part that carries positions; some tokens stand out
        wide = _normal(g, T, c["dc"] + c["dr"], dtype=torch.float32)
        wide *= torch.where(torch.rand((T, 1), device=DEV, generator=g) < 0.02, 50.0, 1.0)
        s["wide"] = wide.bfloat16()
        s["latent"], s["rope"] = torch.zeros((rows, c["dc"]), dtype=torch.bfloat16, device=DEV), torch.zeros((rows, c["dr"]), dtype=torch.bfloat16, device=DEV)
        return s
    s["scale"] = (c["hd"] + c["dr"]) ** -0.5
    width = c["dc"] if c["op"] == "absorbed" else c["hd"]
    s["q"] = _normal(g, T, c["H"], width + c["dr"])
    s["out"] = torch.zeros((T, c["H"], width), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((T, c["H"]), dtype=torch.float32, device=DEV)
    if c["op"] == "absorbed":
        s["pool"] = _pool(s, g)
        return s
    new, held = _lens(c)
    lens = torch.where(new > 0, new + held, 0)
    s["row_start"] = torch.cat([lens.new_zeros(1), torch.cumsum(lens, 0)]).to(torch.int32).to(DEV)
    rows = int(lens.sum())
    s["kv"], s["k_rope"] = _normal(g, rows, c["H"], 2 * c["hd"]), _normal(g, rows, c["dr"])
    return s


# ---------------------------------------------------------------- plain forms


def _rows(c, latent, rope):
    """Cache rows of latents and rotary parts [n, .]: bf16 side by side; or e4m3 codes, 16 bytes of
    exponents (one for 32 features: the least that keeps their magnitudes within 448), bf16."""
    if not c["fp8"]:
        return torch.cat([latent, rope], -1)
    n, dc = latent.shape
    x = latent.float().view(n, dc // 32, 32)
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, m in [1/2, 1)
    byte = (e - 9 + (m > 0.875) + 127).clamp(min=0)
    byte = torch.where(top > 0, byte, 0).to(torch.int32)
    up = ((254 - byte) << 23).view(torch.float32)  # 2^(127 - byte)
    codes = (x * up[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, dc)
    exps = torch.zeros((n, 16), dtype=torch.uint8, device=latent.device)
    exps[:, : dc // 32] = byte.to(torch.uint8)
    return torch.cat([codes, exps, rope.contiguous().view(torch.uint8)], -1)


def _values(c, rows):
    """Latents [..., dc] and rotary parts [..., dr] in 32 bits of cache rows."""
    dc, dr = c["dc"], c["dr"]
    if not c["fp8"]:
        return rows[..., :dc].float(), rows[..., dc:].float()
    codes = rows[..., :dc].contiguous().view(torch.float8_e4m3fn).float()
    byte = rows[..., dc: dc + dc // 32].to(torch.int32)
    down = torch.where(byte > 0, byte << 23, 0x00400000).view(torch.float32)  # 2^(byte - 127)
    latent = (codes.unflatten(-1, (dc // 32, 32)) * down[..., None]).flatten(-2)
    return latent, rows[..., dc + 16:].contiguous().view(torch.bfloat16).float()


def _plain_cache(s):
    p, bs = s["plan"], s["block"]
    flat = s["pool"].view(s["n_blocks"] * bs, -1)
    fresh = _rows(s, s["wide"][:, : s["dc"]], s["wide"][:, s["dc"]:])
    used = p["slots"] >= 0
    flat[p["slots"][used]] = fresh[used]
    start = p["token_start"].long()
    lens = torch.where(start[1:] > start[:-1], p["seq_lens"].long(), 0)
    first = torch.cat([lens.new_zeros(1), torch.cumsum(lens, 0)])
    i = torch.arange(s["latent"].shape[0], device=DEV)
    r = torch.searchsorted(first[1:], i, right=True)
    at = i - first[r]
    latent, rope = _values(s, flat[s["table"][r, at // bs].long() * bs + at % bs])
    s["latent"].copy_(latent)
    s["rope"].copy_(rope)
    return {"latent": s["latent"], "rope": s["rope"], "row_start": first.to(torch.int32)}


def _attend(s, q, k, v, pos, n_keys):
    """softmax(scale q k^T) v over the visible keys in 32 bits, and the logarithm of the softmax's sum:
    q [R, Q, h, D] or k [R, S, D] shared by the heads; key j of a request stands at position j."""
    R, Q, H, D = q.shape
    S = k.shape[1]
    shared = k.dim() == 3
    if shared:
        z = torch.matmul(q.reshape(R, Q * H, D), k.transpose(1, 2).contiguous()).view(R, Q, H, S)
    else:
        z = torch.matmul(q.transpose(1, 2).contiguous(), k.permute(0, 2, 3, 1).contiguous()).transpose(1, 2)
    z = z * s["scale"]
    j = torch.arange(S, device=DEV)
    seen = (j <= pos[..., None]) & (j < n_keys[:, None, None])
    if s["window"]:
        seen &= j > pos[..., None] - s["window"]
    z = z.masked_fill_(~seen[:, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    z = z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    if shared:
        o = torch.matmul(z.reshape(R, Q * H, S), v).view(R, Q, H, -1)
    else:
        o = torch.matmul(z.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()).transpose(1, 2)
    o = torch.where(total > 0, o / total, 0.0)
    return o, (top + total.log()).squeeze(-1)


def _plain_attention(s):
    p = s["plan"]
    new, held = _lens(s)
    Q, S = int(new.max()), int((new + held)[new > 0].max())
    start = p["token_start"].long()
    i = torch.arange(Q, device=DEV)
    count = start[1:] - start[:-1]
    token = (start[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].float()[token]
    pos = p["start_pos"].long()[:, None] + i
    j = torch.arange(S, device=DEV)
    if s["op"] == "absorbed":
        bs = s["block"]
        flat = s["pool"].view(s["n_blocks"] * bs, -1)
        entry = (j // bs).clamp(max=s["max_blocks"] - 1)
        c, kr = _values(s, flat[s["table"][:, entry].long() * bs + j % bs])
        o, lse = _attend(s, q, torch.cat([c, kr], -1), c, pos, p["seq_lens"].long())
    else:
        hd = s["hd"]
        first = s["row_start"].long()
        rows = (first[:-1, None] + j).clamp(max=s["kv"].shape[0] - 1)
        kv, kr = s["kv"].float()[rows], s["k_rope"].float()[rows]
        k = torch.cat([kv[..., :hd], kr[:, :, None].expand(-1, -1, s["H"], -1)], -1)
        o, lse = _attend(s, q, k, kv[..., hd:], pos, first[1:] - first[:-1])
    used = i < count[:, None]
    s["out"][token[used]] = o[used].to(torch.bfloat16)
    s["lse"][token[used]] = lse[used]
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the package's calls


def _handle(s):
    """What a program keeps beside its tensors: the layouts and the plan's buffers."""
    import hashed_gram_engram_amd as eg
    plan = eg.BatchPlan(s["R"], s["T"], device=DEV)
    for name, t in s["plan"].items():
        getattr(plan, name).copy_(t)
    lay = eg.make_latent_layout(s.get("H", 1), s.get("dc", 512), s["dr"], head_dim=s.get("hd", 128), scale=s.get("scale", 1.0),
                                window=s.get("window", 0), cache_format=eg.CACHE_MXFP8 if s.get("fp8") else eg.CACHE_BF16)
    pages = eg.make_page_layout(s["block"], s["max_blocks"], s["n_blocks"]) if "block" in s else None
    return eg, lay, pages, plan


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    eg, lay, pages, plan = s["handle"]
    if s["op"] == "cache":
        eg.engram_latent_write(lay, pages, s["wide"][:, : s["dc"]], s["wide"][:, s["dc"]:], plan, s["pool"])
        latent, rope, first = eg.engram_latent_read(lay, pages, s["pool"], plan, s["table"], s["latent"].shape[0], latent=s["latent"], rope=s["rope"])
        return {"latent": latent, "rope": rope, "row_start": first}
    if s["op"] == "absorbed":
        out = eg.engram_latent_attention(lay, pages, s["q"], s["pool"], plan, s["table"], out=s["out"], lse=s["lse"])
    else:
        out = eg.engram_latent_attention_expanded(lay, s["q"], s["kv"], s["k_rope"], s["row_start"], plan, out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return _plain_cache(state) if state["op"] == "cache" else _plain_attention(state)


# ---------------------------------------------------------------- floors and exact results


def work(case):
    c = case
    new, held = _lens(c)
    on = new > 0
    new, held = new[on].double(), held[on].double()
    T = float(new.sum())
    row = 2 * ((c.get("dc", 0)) + c["dr"])  # of the cache
    if c.get("fp8"):
        row = c["dc"] + c["dc"] // 32 + 2 * c["dr"]
    if c["op"] == "cache":
        wide, rows = 2 * (c["dc"] + c["dr"]), float((new + held).sum())
        return {"bytes": T * (wide + row) + rows * (row + wide), "flops": 0}
    w = c["window"] or 1 << 40
    # the token at position p sees min(p + 1, w) keys; a request reads the keys that any of its tokens sees
    full = (held + new).clamp(max=w)
    few = (held + 1).clamp(max=w)
    short = full - few  # tokens, but one, that see one key more than the last did
    pairs = float((few * (short + 1) + short * (short + 1) / 2 + (new - 1 - short) * full).sum())
    keys = float(torch.minimum(held + new, w + new - 1).sum())
    H = c["H"]
    if c["op"] == "absorbed":
        return {"bytes": keys * row + T * H * (2 * (2 * c["dc"] + c["dr"]) + 4), "flops": pairs * H * 2 * (2 * c["dc"] + c["dr"])}
    return {"bytes": keys * 2 * (2 * c["hd"] * H + c["dr"]) + T * H * (2 * (2 * c["hd"] + c["dr"]) + 4),
            "flops": pairs * H * 2 * (2 * c["hd"] + c["dr"])}


def _power(e):
    """2^e in 64 bits, exactly (pow may be off in its last bit, which moves ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rows(c, rows):
    """The latents that cache rows stand for, in 64 bits, from their bits."""
    dc = c["dc"]
    if not c["fp8"]:
        return rows.double()
    b = rows[:, :dc].long()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (8 + m) * _power(e - 10), m * 2.0 ** -9)
    mag = torch.where(b >= 128, -mag, mag) * torch.repeat_interleave(_power(rows[:, dc: dc + dc // 32].long() - 127), 32, dim=1)
    return torch.cat([mag, rows[:, dc + 16:].contiguous().view(torch.bfloat16).double()], 1)


def exact(case, seed):
    s = prepare(case, seed)
    new, held = _lens(case)
    start, first = 0, 0
    if s["op"] == "cache":
        latents, ropes, bounds = [], [], [0]
        for r in range(s["R"]):
            n, h = int(new[r]), int(held[r])
            if n:
                j = torch.arange(h, device=DEV)
                old = _exact_rows(s, s["pool"][s["table"][r, j // s["block"]].long(), j % s["block"]])
                x = s["wide"][start: start + n].double()
                c = x[:, : s["dc"]]
                if s["fp8"]:
                    blocks = c.reshape(n, -1, 32)
                    m, e = torch.frexp(blocks.abs().amax(-1, keepdim=True).clamp(min=1e-30) / 448)
                    step = _power(e - (m == 0.5).int())  # the power of two not below the quotient
                    y = blocks / step
                    # e4m3: four significant bits, none below 2^-9
                    ulp = _power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
                    c = (torch.round(y / ulp) * ulp * step).reshape(n, -1)
                both = torch.cat([old, torch.cat([c, x[:, s["dc"]:]], 1)])
                latents.append(both[:, : s["dc"]])
                ropes.append(both[:, s["dc"]:])
                start += n
            bounds.append(bounds[-1] + (n + h if n else 0))
        return {"latent": torch.cat(latents), "rope": torch.cat(ropes), "row_start": torch.tensor(bounds, dtype=torch.int32, device=DEV)}
    out, lse = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for r in range(s["R"]):
        n, h = int(new[r]), int(held[r])
        if n == 0:
            continue
        q = s["q"][start: start + n].double()
        j, p = torch.arange(h + n, device=DEV), torch.arange(h, h + n, device=DEV)[:, None]
        hidden = (j > p) | (j <= p - (s["window"] or 1 << 40))
        if s["op"] == "absorbed":
            k = _exact_rows(s, s["pool"][s["table"][r, j // s["block"]].long(), j % s["block"]])
        for a in range(s["H"]):
            if s["op"] == "absorbed":
                v = k[:, : s["dc"]]
            else:
                kv = s["kv"][first: first + h + n, a].double()
                k, v = torch.cat([kv[:, : s["hd"]], s["k_rope"][first: first + h + n].double()], 1), kv[:, s["hd"]:]
            z = (torch.mm(q[:, a], k.t().contiguous()) * s["scale"]).masked_fill(hidden, -math.inf)
            lse[start: start + n, a] = torch.logsumexp(z, 1)
            out[start: start + n, a] = torch.mm(torch.softmax(z, 1), v)
        start += n
        first += h + n
    return {"out": out, "lse": lse}
