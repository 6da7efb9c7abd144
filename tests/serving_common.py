"""Plain implementations of the serving operators, written from their formulas: the plan and the paged
hash as scalar Python over one request and one token at a time, the norms and the product in 64 bits."""
import math

import numpy as np
import torch

import oracle

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value
U = 2.0 ** -24                                                  # half a step of fp32


def plan_ref(block_size, max_blocks, n_blocks, new, held, table, free, count, max_tokens):
    """The plan of one step: a dict of the plan's fields, the table and list after it, and the errors
    counted."""
    R, bs, cap = len(new), block_size, block_size * max_blocks
    new, held = [int(v) for v in new], [int(v) for v in held]
    table, free = table.copy(), free.copy()
    stack = list(free[: min(max(int(count), 0), n_blocks)])
    status, seq, errors = [0] * R, list(held), 0

    def pages(n):
        return -(-n // bs)

    for r in range(R):
        if not 0 <= held[r] <= cap or (new[r] > 0 and held[r] + new[r] > cap):
            status[r] = 3
        elif new[r] < 0:
            seq[r] = 0
            for b in range(pages(held[r])):
                if len(stack) < n_blocks:
                    free[len(stack)] = table[r, b]
                    stack.append(table[r, b])
                else:
                    errors += 1
    avail, asked, needed = len(stack), 0, 0
    start, slots, positions, requests = [0], [], [], []
    for r in range(R):
        n = 0
        if status[r] == 0 and new[r] > 0:
            asked += new[r]
            if asked > max_tokens:
                status[r] = 1
            else:
                more = pages(held[r] + new[r]) - pages(held[r])
                needed += more
                if more > 0 and needed > avail:
                    status[r] = 2
                else:
                    n = new[r]
                    seq[r] = held[r] + n
                    for b in range(more):
                        table[r, pages(held[r]) + b] = stack.pop()
        for p in range(held[r], held[r] + n):
            page = int(table[r, p // bs])
            good = 0 <= page < n_blocks
            errors += not good
            slots.append(page * bs + p % bs if good else -1)
            positions.append(p)
            requests.append(r)
        start.append(start[-1] + n)
    errors += sum(s != 0 for s in status)
    pad = [-1] * (max_tokens - len(slots))
    return dict(token_start=start, start_pos=held, seq_lens=seq, status=status, free_left=[len(stack)], slots=slots + pad,
                positions=positions + pad, requests=requests + pad,
                live=[1] * len(slots) + [0] * len(pad)), table, free, errors


def hash_ref(h, ids, mask, plan, block_size, table, history):
    """Row ids [n_layers, n_tokens, n_cols] of a plan's tokens, each request by the sequence oracle with
    its pages laid out as one history; history [n_blocks, block_size] is updated."""
    n = len(ids)
    dead = [np.full((1, 1), 0)]
    pad = oracle.hash_ids(dead[0], h["token_map"].astype(np.int64), h["multipliers"], h["primes"], h["offsets"], h["pad_id"],
                          np.zeros((1, 1), np.int64), start_pos=0, token_mask=np.zeros((1, 1), np.uint8))  # [1, 1, L, C]
    out = np.repeat(pad[0].transpose(1, 0, 2), n, axis=1)
    for r in range(len(plan["start_pos"])):
        a, b, p0 = plan["token_start"][r], plan["token_start"][r + 1], plan["start_pos"][r]
        if a == b:
            continue
        seq = np.zeros((1, p0 + b - a), np.int64)
        for q in range(p0):
            seq[0, q] = history[table[r, q // block_size], q % block_size]
        ref = oracle.hash_ids(ids[None, a:b], h["token_map"].astype(np.int64), h["multipliers"], h["primes"], h["offsets"],
                              h["pad_id"], seq, start_pos=p0, token_mask=None if mask is None else mask[None, a:b])
        out[:, a:b] = ref[0].transpose(1, 0, 2)
        for q in range(p0, p0 + b - a):
            history[table[r, q // block_size], q % block_size] = seq[0, q]
    return out


def norm_ref(x, y, gate, kind, post_w, pre_w, mask, alpha, beta, post_eps, pre_eps, post_norm=True):
    """(out, h, bound of out, bound of h) in 64 bits, from tensors on any device.  Bounds: fp32 sums of
    squares of positive terms, at most 40 in a thread, 6 levels of a tree over a wave and 16 waves one
    after the other, are within 90 u, the root halves that; with the division, root, weight, gate (exp
    within 4 u) and scale a term of n is within 64 u; then two products, a sum and the output's rounding."""
    x64 = x.double().cpu()
    r, dr = x64, torch.zeros_like(x64)
    if y is not None:
        n = y.double().cpu()
        if post_norm:
            n = n / torch.sqrt(n.square().mean(-1, keepdim=True) + post_eps)
        n = n.expand_as(x64)
        if post_w is not None:
            n = n * post_w.double().cpu()
        if kind == "token":
            n = n * gate.double().cpu()[..., None]
        elif kind == "feature":
            n = n * torch.sigmoid(gate.double().cpu())
        s = alpha * x64 + beta * n
        ds = 66 * U * (beta * n).abs() + 3 * U * ((alpha * x64).abs() + (beta * n).abs())
        if mask is not None:
            opened = mask.cpu().bool()[..., None, None].expand_as(x64)
            s, ds = torch.where(opened, s, x64), torch.where(opened, ds, 0.0)
        r, dr = s, ds
    rstd = 1.0 / torch.sqrt(r.square().mean(-1, keepdim=True) + pre_eps)
    w = 1.0 if pre_w is None else pre_w.double().cpu()
    h = r * rstd * w
    # an error of r moves h by itself and, through the mean square, by at most as much again
    dh = (dr + dr.square().mean(-1, keepdim=True).sqrt() * rstd * r.abs()) * rstd * abs(w) + 64 * U * h.abs()
    return r, h, dr + EPS[x.dtype] * (r.abs() + dr), dh + EPS[torch.bfloat16] * (h.abs() + dh)


def act_ref(z, act):
    """act(z) in 64 bits and its largest slope."""
    if act == "relu":
        return z.clamp(min=0), 1.0
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5)), 1.13
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)), 1.13
    if act == "silu":
        return z * torch.sigmoid(z), 1.1
    if act == "sigmoid":
        return torch.sigmoid(z), 0.25
    return z, 1.0


def linear_ref(x, w, bias, res, act, glu, dtype):
    """(out, bound) in 64 bits.  Bound: an fp32 sum of K products is within K 2^-23 of the sum of their
    magnitudes in any order, rounded or truncated; the activation passes that on by its slope and adds
    8 u of its value and of its argument (erf, exp and the division within 4 u each)."""
    xd, wd = x.double().cpu(), w.double().cpu()
    K = xd.shape[-1]
    z, dz = xd @ wd.T, (K + 2) * 2.0 ** -23 * (xd.abs() @ wd.abs().T)
    if bias is not None:
        b = bias.double().cpu()
        z, dz = z + b, dz + 2 * U * (z.abs() + b.abs())
    if glu:
        n = z.shape[-1] // 2
        v, slope = act_ref(z[..., :n], act)
        dv = slope * dz[..., :n] + 8 * U * (v.abs() + z[..., :n].abs())
        u, du = z[..., n:], dz[..., n:]
        out, d = v * u, dv * u.abs() + (v.abs() + dv) * du + U * (v * u).abs()
    else:
        out, slope = act_ref(z, act)
        d = slope * dz + 8 * U * (out.abs() + z.abs())
    if res is not None:
        out = out + res.double().cpu()
    return out, d + U * out.abs() + EPS[dtype] * (out.abs() + d)


def near(got, ref, bound, what=""):
    got = got.double().cpu()
    off = (got - ref).abs()
    worst = (off - bound).max().item()
    assert worst <= 0, f"{what}: {int((off > bound).sum())} of {off.numel()} outside, worst by {worst:.3e}"
