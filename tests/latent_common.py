"""Plain implementations of the latent cache and its attention in 64 bits, one request and one head at a time,
and their bounds."""
import math

import numpy as np
import torch

EPS = 2.0 ** -8  # half a step of bf16, relative to the value
U = 2.0 ** -24   # half a step of fp32


def bits_bf16(t):
    """The bit patterns of a bf16 tensor."""
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def bf16_value(bits):
    with np.errstate(invalid="ignore"):
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_values():
    """The value of each of the 256 e4m3fn codes."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v[c] = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        if c & 127 == 127:
            v[c] = math.nan
        if c & 128:
            v[c] = -v[c]
    return v


def quantise_row(x):
    """(codes, scale bytes) of a row of bf16 values [n], n a multiple of 32: by search, not by bit tricks."""
    grid = e4m3_values()[:127]  # 0 .. 448 ascending
    codes, scales = np.zeros(len(x), np.uint8), np.zeros(len(x) // 32, np.uint8)
    for b in range(len(x) // 32):
        v = x[32 * b: 32 * b + 32]
        top = max([abs(a) for a in v if math.isfinite(a)], default=0.0)
        byte = 1
        while top > 448 * 2.0 ** (byte - 127):
            byte += 1
        scales[b] = byte
        for i, a in enumerate(v):
            if not math.isfinite(a):
                codes[32 * b + i] = 0x7F
                continue
            y = abs(a) * 2.0 ** (127 - byte)
            k = int(np.searchsorted(grid, y))
            if byte == 247 and y > 240:
                k = 119  # the next code, 256, stands for 2^128, which bf16 has not
            elif k == 127 or (k > 0 and (y - grid[k - 1] < grid[k] - y or (y - grid[k - 1] == grid[k] - y and k % 2 == 1))):
                k -= 1  # to nearest, ties to the even code
            codes[32 * b + i] = k | (0x80 if math.copysign(1.0, a) < 0 else 0)
    return codes, scales


def row_bytes(dc, dr, fp8):
    return dc + 16 + 2 * dr if fp8 else 2 * (dc + dr)


def make_rows(latent_bits, rope_bits, fp8):
    """Cache rows [n, bytes] of bf16 bit patterns."""
    n, dc = latent_bits.shape
    if not fp8:
        return np.concatenate([latent_bits, rope_bits], 1).view(np.uint8)
    out = np.zeros((n, row_bytes(dc, rope_bits.shape[1], True)), np.uint8)
    for i in range(n):
        out[i, :dc], out[i, dc: dc + dc // 32] = quantise_row(bf16_value(latent_bits[i]))
    out[:, dc + 16:] = rope_bits.view(np.uint8).reshape(n, -1)
    return out


def row_values(rows, dc, fp8):
    """(latents, rope parts) in 64 bits of cache rows [n, bytes]."""
    rows = np.ascontiguousarray(rows)
    if not fp8:
        v = bf16_value(rows.view(np.uint16))
        return v[:, :dc], v[:, dc:]
    scale = 2.0 ** (rows[:, dc: dc + dc // 32].astype(np.float64) - 127)
    scale[rows[:, dc: dc + dc // 32] == 255] = math.nan
    latent = e4m3_values()[rows[:, :dc]] * np.repeat(scale, 32, 1)
    return latent, bf16_value(np.ascontiguousarray(rows[:, dc + 16:]).view(np.uint16))


def attend_ref(q, k, v, pos, key_pos, scale, window, alive=None):
    """(out, lse, bound of out, bound of lse) in 64 bits of one head: q [n, D], k [m, D], v [m, E] as numpy, token i
    at pos[i], key j at key_pos[j].

    Bounds: a score is an fp32 sum of D products, within (D + 2) 2^-23 of the sum of their magnitudes, times the
    scale; with the scale and log2 e (rounded once each), the difference to the reference maximum (two roundings of
    values within |s| + |m|) and 2^x within 4 u, a weight is off by that much relative.  Weights are rounded to bf16
    for the second product only; sums over m keys of positive terms add m 2^-23, and up to two rescalings and joins
    8 u.  The output is rounded to bf16 once."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n, m = q.shape[0], k.shape[0]
    seen = key_pos[None, :] <= pos[:, None]
    if window:
        seen &= key_pos[None, :] > pos[:, None] - window
    if alive is not None:
        seen &= alive[None, :]
    out, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    d_out, d_lse = np.zeros_like(out), np.zeros(n)
    for i in range(n):
        j = np.nonzero(seen[i])[0]
        if len(j) == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * (k[j] @ q[i])
            mag = abs(scale) * (np.abs(k[j]) @ np.abs(q[i]))
            top = s.max()
            p = np.exp(s - top)
            total = p.sum()
            out[i], lse[i] = p @ v[j] / total, top + math.log(total) if total > 0 else math.nan
            ds = ((q.shape[1] + 2) * 2.0 ** -23 * mag + 8 * U * (np.abs(s) + abs(top) + 16)).max() + 4 * U
            rel = ds + (len(j) + 32) * 2.0 ** -23
            A = p @ np.abs(v[j]) / total
            d = A * (EPS + 2 * rel) * (1 + 2.0 ** -6)  # (second order in the last factor)
            d_out[i] = d + EPS * (np.abs(out[i]) + d)
            d_lse[i] = rel * (1 + 2.0 ** -6) + 4 * U * abs(lse[i])
    return out, lse, d_out, d_lse


def near(got, ref, bound, what=""):
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - ref) <= bound)
        worst = np.nanmax(np.where(same, -np.inf, np.abs(got - ref) - bound)) if got.size else 0
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} outside, worst by {worst:.3e}"


class Step:
    """A step of ragged requests in a shuffled pool, by hand: new and held tokens of each request."""

    def __init__(self, new, held, block, rng, max_tokens=None, spare=3, max_blocks=None):
        self.new, self.held, self.block = [int(v) for v in new], [int(v) for v in held], block
        R = len(new)
        self.R = R
        need = [-(-(n + h) // block) for n, h in zip(self.new, self.held)]
        self.max_blocks = max_blocks or max(1, max(need))
        self.n_blocks = sum(need) + spare
        order = rng.permutation(self.n_blocks).astype(np.int32)
        self.table = np.full((R, self.max_blocks), -1, np.int32)
        at = 0
        for r in range(R):
            self.table[r, : need[r]] = order[at: at + need[r]]
            at += need[r]
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        live = int(self.start[-1])
        self.T = live if max_tokens is None else max_tokens
        self.slots = np.full(self.T, -1, np.int64)
        for r in range(R):
            for i in range(self.new[r]):
                p = self.held[r] + i
                self.slots[self.start[r] + i] = int(self.table[r, p // block]) * block + p % block

    def slot_list(self, r, lo, hi):
        p = np.arange(lo, hi)
        page = self.table[r, p // self.block].astype(np.int64)
        s = page * self.block + p % self.block
        return np.where((page >= 0) & (page < self.n_blocks), s, -1)

    def plan(self, eg, device="cuda"):
        plan = eg.BatchPlan(self.R, self.T, device=device)
        plan.token_start.copy_(torch.from_numpy(self.start))
        plan.start_pos.copy_(torch.tensor(self.held, dtype=torch.int32))
        plan.seq_lens.copy_(torch.tensor(self.held, dtype=torch.int32) + torch.tensor(self.new, dtype=torch.int32))
        plan.slots.copy_(torch.from_numpy(self.slots))
        return plan

    def pages(self, eg):
        return eg.make_page_layout(self.block, self.max_blocks, self.n_blocks)

    def table_on(self, device="cuda"):
        return torch.from_numpy(self.table).to(device)


def cache_on(rows, dc, dr, fp8, step, device="cuda"):
    """Rows [n_blocks * block, bytes] as the cache tensor."""
    t = torch.from_numpy(rows).to(device)
    return t.view(step.n_blocks, step.block, -1) if fp8 else t.view(torch.bfloat16).view(step.n_blocks, step.block, dc + dr)
