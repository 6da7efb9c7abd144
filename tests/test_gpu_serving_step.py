"""Serving steps of ragged requests through the operators together: plan -> paged hash -> engram_forward ->
norm -> gated product -> product with the residual stream -> norm with gate, over a prompt step, decode
steps and a step in which requests finish.  Row ids must equal engram_hash_ids on each request's own
sequence, the forward its output on those ids bit for bit, and every operator its 64-bit formula on the
inputs it had; one captured graph of a whole step must repeat the eager step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import synth  # noqa: E402
from gpu_common import eg, layout, say  # noqa: E402
from serving_common import linear_ref, near, norm_ref, plan_ref  # noqa: E402

W = synth.get("tiny")
HC, DIM, INNER, R, TOKENS, BLOCK, PAGES = W.hc, W.dim, 328, 6, 61, 8, 60


def cuda(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


class Model:
    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(7)

        def normal(*shape, std=1.0):
            return torch.empty(shape, device="cuda").normal_(0, std, generator=g)
        self.h = synth.hash_inputs(51, 1, 1, n_layers=1, n_heads=2, vocab=700, compressed_vocab=500, primes=[W.primes])
        self.hash = [cuda(self.h[k]) for k in ("token_map", "multipliers", "primes", "offsets")]
        d = synth.device_inputs(W)
        self.engram = [d[k] for k in ("table", "scales", "wkv", "q_weight", "k_weight")]
        self.up, self.up_bias = normal(2 * INNER, DIM, std=DIM ** -0.5).bfloat16(), normal(2 * INNER)
        self.down = normal(DIM, INNER, std=INNER ** -0.5).bfloat16()
        self.pre, self.post = 1 + 0.1 * normal(HC, DIM), 1 + 0.1 * normal(HC, DIM)
        self.embed = normal(700, HC, DIM).bfloat16()
        self.pages = eg.make_page_layout(BLOCK, 12, PAGES)
        self.hl = eg.make_hash_layout(1, 4, 2, self.h["pad_id"], 700, 96)
        self.first = eg.make_norm_layout(HC, DIM, pre_eps=1e-6)
        self.last = eg.make_norm_layout(HC, DIM, gate=eg.GATE_TOKEN, beta=0.5, post_eps=1e-6, pre_eps=1e-6)
        self.gated = eg.make_linear_layout(DIM, INNER, activation=eg.ACT_SILU, glu=True)
        self.plain = eg.make_linear_layout(INNER, DIM)
        self.ws = torch.zeros(max(256, eg.engram_forward_workspace_bytes(layout(W), 1, TOKENS)), dtype=torch.uint8, device="cuda")

    def step(self, s, plan):
        """One step on the state's buffers; what each operator had and gave."""
        eg.engram_batch_plan(self.pages, s["new"], s["held"], s["table"], s["free"], s["count"], plan)
        ids = eg.engram_hash_ids_paged(self.hl, self.pages, *self.hash, s["ids"], plan, s["table"], s["history"])
        x = self.embed[s["ids"]][None]
        live = plan.live[None]
        x1 = eg.engram_forward(layout(W), x, ids[0][None], live, *self.engram, workspace=self.ws)
        _, h = eg.engram_residual_norm(self.first, x1, pre_weight=self.pre)
        u = eg.engram_linear(self.gated, h, self.up, bias=self.up_bias)
        y = eg.engram_linear(self.plain, u, self.down, residual=h)
        gate = s["gate"]
        out, h2 = eg.engram_residual_norm(self.last, x1, y, gate=gate, post_weight=self.post, pre_weight=self.pre, token_mask=live)
        return dict(ids=ids, x=x, x1=x1, h=h, u=u, y=y, out=out, h2=h2)


def test_steps_of_ragged_requests():
    say("[gpu] serving steps: a prompt step, decode steps, finished requests")
    m, rng = Model(), np.random.default_rng(3)
    table, free = np.full((R, 12), -1, np.int32), rng.permutation(PAGES).astype(np.int32)
    held, count = np.zeros(R, np.int32), PAGES
    s = dict(table=cuda(table), free=cuda(free), history=torch.zeros((PAGES, BLOCK), dtype=torch.int64, device="cuda"))
    texts = [[] for _ in range(R)]
    plan = eg.BatchPlan(R, TOKENS)
    for new in ([20, 1, 13, 0, 9, 18], [1] * 6, [1, 1, -1, 30, 1, 1], [1, 40, 7, 1, 1, -1], [1, 1, 1, 1, 1, 5]):
        ref, table, free, errors = plan_ref(BLOCK, 12, PAGES, new, held, table, free, count, TOKENS)
        assert errors == 0
        ids = rng.integers(0, 700, TOKENS)
        s |= dict(new=cuda(np.array(new, np.int32)), held=cuda(held), count=cuda(np.array([count], np.int32)), ids=cuda(ids),
                  gate=torch.rand((1, TOKENS, HC), device="cuda"))
        got = m.step(s, plan)
        for f in eg.BatchPlan.FIELDS:
            assert np.array_equal(getattr(plan, f).cpu().numpy(), np.array(ref[f])), f
        # row ids: each request's whole text through engram_hash_ids
        want = got["ids"].clone()
        for r in range(R):
            a, b = ref["token_start"][r], ref["token_start"][r + 1]
            texts[r] = [] if new[r] < 0 else texts[r] + ids[a:b].tolist()
            if a < b:
                t = torch.tensor([texts[r]], dtype=torch.int64, device="cuda")
                hist = torch.zeros((1, 96), dtype=torch.int64, device="cuda")
                want[:, a:b] = eg.engram_hash_ids(m.hl, *m.hash, t, hist)[:, 0, len(texts[r]) - (b - a):]
        assert torch.equal(got["ids"], want)
        live = plan.live[None]
        x1 = eg.engram_forward(layout(W), got["x"], want[0][None].contiguous(), live, *m.engram, check=True)
        assert torch.equal(got["x1"], x1) and torch.equal(x1[~live.bool()], got["x"][~live.bool()])
        _, hr, _, bh = norm_ref(x1, None, None, "none", None, m.pre, None, 1, 1, 0, 1e-6)
        near(got["h"], hr, bh, "h")
        flat = got["h"].view(-1, DIM)
        near(got["u"].view(-1, INNER), *linear_ref(flat, m.up, m.up_bias, None, "silu", True, torch.bfloat16), "gated")
        near(got["y"].view(-1, DIM), *linear_ref(got["u"].view(-1, INNER), m.down, None, flat, "none", False, torch.bfloat16), "y")
        r, hr, br, bh = norm_ref(x1, got["y"], s["gate"], "token", m.post, m.pre, live, 1.0, 0.5, 1e-6, 1e-6)
        near(got["out"], r, br, "out")
        near(got["h2"], hr, bh, "h2")
        held, count = np.array(ref["seq_lens"], np.int32), ref["free_left"][0]


def test_a_captured_step_repeats_the_eager_one():
    say("[gpu] serving steps: one graph of a whole step, replayed with new tokens")
    m, rng = Model(), np.random.default_rng(4)
    s = dict(table=torch.full((R, 12), -1, dtype=torch.int32, device="cuda"), free=cuda(rng.permutation(PAGES).astype(np.int32)),
             history=torch.zeros((PAGES, BLOCK), dtype=torch.int64, device="cuda"), new=cuda(np.ones(R, np.int32)),
             held=torch.zeros(R, dtype=torch.int32, device="cuda"), count=cuda(np.array([PAGES], np.int32)),
             ids=cuda(rng.integers(0, 700, TOKENS)), gate=torch.rand((1, TOKENS, HC), device="cuda"))
    plan = eg.BatchPlan(R, TOKENS)
    eager = {k: v.clone() for k, v in s.items()}
    eager_plan = eg.BatchPlan(R, TOKENS)
    m.step(s, plan)
    for k in ("table", "free", "history"):  # back to the start
        s[k].copy_(eager[k])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.step(s, plan)
        s["held"].copy_(plan.seq_lens)  # the next step goes on from here
        s["count"].copy_(plan.free_left)
    for k in range(20):  # past several pages of 8
        ids = torch.from_numpy(rng.integers(0, 700, TOKENS)).cuda()
        s["ids"].copy_(ids)
        eager["ids"].copy_(ids)
        graph.replay()
        want = m.step(eager, eager_plan)
        eager["held"].copy_(eager_plan.seq_lens)
        eager["count"].copy_(eager_plan.free_left)
        torch.cuda.synchronize()
        assert int(plan.seq_lens[0]) == k + 1
        for name in got:
            assert torch.equal(got[name], want[name]), (k, name)
        for name in ("table", "free", "history", "held", "count"):
            assert torch.equal(s[name], eager[name]), (k, name)
