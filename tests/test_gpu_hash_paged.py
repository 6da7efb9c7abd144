"""engram_hash_ids_paged against the sequence oracle, request by request: exact row ids and history over
ragged steps, dead spans, bad ids and pages, and the tokens behind the last."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import synth  # noqa: E402
from gpu_common import eg, say  # noqa: E402
from serving_common import hash_ref, plan_ref  # noqa: E402


def cuda(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


class Server:
    """A host copy and a device copy of one pool, stepped together."""

    def __init__(self, h, R, block, max_blocks, n_blocks, max_tokens, seed=0):
        rng = np.random.default_rng(seed)
        self.h, self.block, self.R, self.max_tokens = h, block, R, max_tokens
        self.lay = eg.make_page_layout(block, max_blocks, n_blocks)
        self.hl = eg.make_hash_layout(h["n_layers"], h["max_ngram"], h["n_heads"], h["pad_id"], h["vocab"], max_blocks * block)
        self.table = np.full((R, max_blocks), -1, np.int32)
        self.free = rng.permutation(n_blocks).astype(np.int32)
        self.count, self.held = n_blocks, np.zeros(R, np.int32)
        self.history = rng.integers(0, 50, (n_blocks, block))
        self.dev = dict(table=cuda(self.table), free=cuda(self.free), history=cuda(self.history))
        self.plan = eg.BatchPlan(R, max_tokens)
        self.args = [cuda(h["token_map"]), cuda(h["multipliers"]), cuda(h["primes"]), cuda(h["offsets"])]

    def step(self, new, ids, mask):
        ref, self.table, self.free, _ = plan_ref(self.block, self.lay.max_blocks, self.lay.n_blocks, new, self.held, self.table,
                                                 self.free, self.count, self.max_tokens)
        d = self.dev
        eg.engram_batch_plan(self.lay, cuda(np.array(new, np.int32)), cuda(self.held), d["table"], d["free"],
                             cuda(np.array([self.count], np.int32)), self.plan)
        got = eg.engram_hash_ids_paged(self.hl, self.lay, *self.args, cuda(ids), self.plan, d["table"], d["history"],
                                       token_mask=None if mask is None else cuda(mask))
        want = hash_ref(self.h, ids, mask, ref, self.block, self.table, self.history)
        self.held, self.count = np.array(ref["seq_lens"], np.int32), ref["free_left"][0]
        assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(d["history"].cpu().numpy(), self.history)
        return ref


@pytest.mark.parametrize("block,layers,ngram,heads", [(16, 2, 4, 8), (1, 1, 2, 1), (7, 3, 8, 5), (64, 2, 3, 100)])
def test_ragged_steps_match_the_sequence_oracle(block, layers, ngram, heads):
    say(f"[gpu] paged hash: pages of {block}, {layers} layers, {ngram}-grams, {heads} heads")
    h = synth.hash_inputs(41, 1, 1, n_layers=layers, max_ngram=ngram, n_heads=heads, vocab=3000, compressed_vocab=2000,
                          primes=[synth.primes_from(1009 + 500 * y, (ngram - 1) * heads) for y in range(layers)])
    s = Server(h, 9, block, -(-400 // block), 9 * -(-400 // block), 300, seed=block)
    rng = np.random.default_rng(block)
    for step in range(6):
        new = rng.integers(0, 3, 9) if step % 2 else rng.integers(0, 60, 9)
        new = np.where(rng.random(9) < 0.1, -1, new)
        if step == 0:
            new = np.array([1, 2, 3, 4, 0, 5, 60, 33, 7])
        ids = rng.integers(0, 3000, 300)
        mask = (rng.random(300) > 0.1).astype(np.uint8) if step != 3 else None
        s.step(new, ids, mask)


def test_many_tokens_at_the_model_sizes():
    say("[gpu] paged hash: 5000 tokens of 17 requests at the model's sizes")
    h = synth.hash_inputs(42, 1, 1)
    s = Server(h, 17, 24, 50, 17 * 50, 5003)
    rng = np.random.default_rng(3)
    for new in (rng.integers(100, 400, 17), rng.integers(1, 300, 17)):
        ref = s.step(new, rng.integers(0, h["vocab"], 5003), (rng.random(5003) > 0.02).astype(np.uint8))
        assert ref["live"][-1] == 0


def test_signed_extremes_and_large_primes():
    say("[gpu] paged hash: extreme products and primes up to 2^62")
    h = synth.hash_inputs(43, 1, 1, n_layers=1, max_ngram=3, n_heads=4, vocab=500, compressed_vocab=400,
                          primes=[[1, 2, 3, 2 ** 31 - 1, 2 ** 61 - 1, 2 ** 62 - 57, 16000057, 5]])
    h["multipliers"] = np.array([[-2 ** 63 + 1, 2 ** 63 - 1, -1]], np.int64)
    h["offsets"] = np.zeros_like(h["offsets"])
    s = Server(h, 2, 8, 64, 128, 700)
    s.step([400, 300], np.random.default_rng(0).integers(0, 500, 700), None)


def test_bad_ids_pages_and_plans_are_dead_and_counted():
    say("[gpu] paged hash: ids outside the map, pages outside the pool, requests outside the plan")
    h = synth.hash_inputs(44, 1, 1, n_layers=1, vocab=100, compressed_vocab=100)
    lay = eg.make_page_layout(4, 4, 8)
    hl = eg.make_hash_layout(1, 4, 8, 2, 100, 16)
    table = np.array([[0, 1, 2, 3], [9, -1, 4, 5]], np.int32)
    history = np.arange(32).reshape(8, 4)
    plan = eg.BatchPlan(2, 7)
    plan.start_pos.copy_(torch.tensor([3, 5]))
    plan.requests.copy_(torch.tensor([0, 0, 0, 1, 2, -1, 1]))
    plan.positions.copy_(torch.tensor([3, 4, 5, 5, 0, -1, 40]))
    plan.slots.copy_(torch.tensor([3, 4, 5, 32, 9, -1, -1]))
    ids = np.array([7, -1, 100, 8, 11, 12, 13])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hist = cuda(history)
    got = eg.engram_hash_ids_paged(hl, lay, cuda(h["token_map"]), cuda(h["multipliers"]), cuda(h["primes"]), cuda(h["offsets"]),
                                   cuda(ids), plan, cuda(table), hist, err_count=err).cpu().numpy()
    want_hist = history.copy()
    want_hist[0, 3], want_hist[1, 0], want_hist[1, 1] = h["token_map"][7], -1, -1
    assert np.array_equal(hist.cpu().numpy(), want_hist)
    # ids -1 and 100; look-backs 1..3 of token 3 (positions 4, 3, 2: entries 1, 0, 0).  The last token's
    # look-backs are all positions of this call
    assert int(err.item()) == 2 + 3

    def row(toks):
        m = h["multipliers"][0].astype(object)
        out, blocked, v = [], False, 0
        for i, t in enumerate(toks):
            blocked = blocked or t < 0
            v ^= (int(2 if blocked else t) * int(m[i])) % 2 ** 64
            if i:
                s = v - 2 ** 64 if v >= 2 ** 63 else v
                out += [s % int(p) + int(o) for p, o in zip(h["primes"][0, i - 1], h["offsets"][0, 8 * (i - 1):8 * i])]
        return out

    t = [int(v) for v in h["token_map"]]
    pads = [-1, -1, -1, -1]
    for i, toks in enumerate([[t[7], 2, 1, 0], [-1, t[7], 2, 1], [-1, -1, t[7], 2], [t[8], -1, -1, -1], pads, pads,
                              [t[13], t[12], t[11], t[8]]]):
        assert got[0, i].tolist() == row(toks), i


def test_history_past_32_bit_offsets():
    say("[gpu] paged hash: history entries past 2^29 (4 GiB)")
    h = synth.hash_inputs(45, 1, 1, n_layers=1, vocab=300, compressed_vocab=300)
    lay = eg.make_page_layout(1 << 20, 2, 600)  # 4.7 GiB
    hl = eg.make_hash_layout(1, 4, 8, 2, 300, 2 << 20)
    history = torch.zeros((600, 1 << 20), dtype=torch.int64, device="cuda")
    table = torch.tensor([[599, 598]], dtype=torch.int32, device="cuda")
    ids = np.random.default_rng(1).integers(0, 300, 12)
    plan = eg.BatchPlan(1, 6)
    parts = []
    for p0 in (0, 6):
        plan.start_pos.fill_(p0)
        plan.requests.zero_()
        plan.positions.copy_(torch.arange(p0, p0 + 6))
        plan.slots.copy_(599 * (1 << 20) + torch.arange(p0, p0 + 6))
        parts.append(eg.engram_hash_ids_paged(hl, lay, cuda(h["token_map"]), cuda(h["multipliers"]), cuda(h["primes"]),
                                              cuda(h["offsets"]), cuda(ids[p0:p0 + 6]), plan, table, history))
    import oracle
    ref = oracle.hash_ids(ids[None], h["token_map"].astype(np.int64), h["multipliers"], h["primes"], h["offsets"], 2,
                          np.zeros((1, 12), np.int64))
    assert np.array_equal(torch.cat(parts, 1).cpu().numpy(), ref[0].transpose(1, 0, 2))
    assert history[:599].abs().sum().item() == 0
