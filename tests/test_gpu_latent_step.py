"""Serving steps through the latent operators as one layer of a model uses them: plan -> projection -> write; requests with
few new tokens by the absorbed form, those with many by read -> product -> expanded form.  Prompts, decoding,
drafts and finished requests; one captured graph of a whole step must repeat the eager step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from latent_common import attend_ref, bits_bf16, make_rows, near, row_values  # noqa: E402

R, TOKENS, BLOCK, PAGES, TABLE, ROWS = 6, 150, 16, 70, 14, 400
H, DC, DR, HD, DIM, FEW = 12, 128, 32, 64, 256, 4


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """One attention layer over the latent cache, with bf16 weights."""

    def __init__(self, fp8, window):
        g = torch.Generator(device="cuda").manual_seed(9)

        def normal(*shape, std=1.0):
            return torch.empty(shape, device="cuda").normal_(0, std, generator=g).bfloat16()
        self.fp8, self.window = fp8, window
        self.lay = eg.make_latent_layout(H, DC, DR, head_dim=HD, window=window, cache_format=eg.CACHE_MXFP8 if fp8 else eg.CACHE_BF16)
        self.scale = float(np.float32(self.lay.scale))
        self.pages = eg.make_page_layout(BLOCK, TABLE, PAGES)
        self.down = normal(DC + DR, DIM, std=DIM ** -0.5)
        self.wq = normal(H * (HD + DR), DIM, std=DIM ** -0.5)
        self.up = normal(H * 2 * HD, DC, std=DC ** -0.5)
        self.to_rows = eg.make_linear_layout(DIM, DC + DR)
        self.to_q = eg.make_linear_layout(DIM, H * (HD + DR))
        self.to_kv = eg.make_linear_layout(DC, H * 2 * HD)
        self.cache = eg.make_latent_cache(self.lay, self.pages)

    def absorbed_q(self, q):
        """The queries' own parts through each head's keys (a plain product), beside the rope parts."""
        wk = self.up.view(H, 2 * HD, DC)[:, :HD].float()
        own = torch.einsum("thd,hdc->thc", q[..., :HD].float(), wk)
        return torch.cat([own.bfloat16(), q[..., HD:]], -1)

    def step(self, s, plan):
        eg.engram_batch_plan(self.pages, s["new"], s["held"], s["table"], s["free"], s["count"], plan)
        rows = eg.engram_linear(self.to_rows, s["x"], self.down)
        q = eg.engram_linear(self.to_q, s["x"], self.wq).view(TOKENS, H, HD + DR)
        eg.engram_latent_write(self.lay, self.pages, rows[:, :DC], rows[:, DC:], plan, self.cache, err_count=s["err"])
        qa = self.absorbed_q(q)
        s["few"].fill_(7.0)
        s["many"].fill_(7.0)
        s["few_lse"].fill_(7.0)
        s["many_lse"].fill_(7.0)
        eg.engram_latent_attention(self.lay, self.pages, qa, self.cache, plan, s["table"], max_tokens=FEW, out=s["few"], lse=s["few_lse"], err_count=s["err"])
        latent, rope, start = eg.engram_latent_read(self.lay, self.pages, self.cache, plan, s["table"], ROWS, min_tokens=FEW + 1, latent=s["latent"],
                                                    rope=s["rope"], row_start=s["row_start"], err_count=s["err"])
        kv = eg.engram_linear(self.to_kv, latent, self.up).view(ROWS, H, 2 * HD)
        eg.engram_latent_attention_expanded(self.lay, q, kv, rope, start, plan, min_tokens=FEW + 1, out=s["many"], lse=s["many_lse"])
        return dict(rows=rows, q=q, qa=qa, kv=kv)


def state(rng, new):
    bf = torch.bfloat16
    return dict(new=cuda(np.array(new, np.int32)), held=torch.zeros(R, dtype=torch.int32, device="cuda"), table=torch.full((R, TABLE), -1, dtype=torch.int32, device="cuda"),
                free=cuda(rng.permutation(PAGES).astype(np.int32)), count=cuda(np.array([PAGES], np.int32)), err=torch.zeros(1, dtype=torch.int32, device="cuda"),
                x=cuda(rng.normal(size=(TOKENS, DIM)).astype(np.float32)).bfloat16(), few=torch.zeros((TOKENS, H, DC), dtype=bf, device="cuda"),
                many=torch.zeros((TOKENS, H, HD), dtype=bf, device="cuda"), few_lse=torch.zeros((TOKENS, H), device="cuda"),
                many_lse=torch.zeros((TOKENS, H), device="cuda"), latent=torch.zeros((ROWS, DC), dtype=bf, device="cuda"),
                rope=torch.zeros((ROWS, DR), dtype=bf, device="cuda"), row_start=torch.zeros(R + 1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("fp8,window", [(True, 0), (False, 0), (True, 24)])
def test_steps_of_ragged_requests(fp8, window):
    say(f"[gpu] latent serving steps fp8={fp8} window={window}")
    m, rng = Layer(fp8, window), np.random.default_rng(41)
    s, plan = state(rng, [0] * R), eg.BatchPlan(R, TOKENS)
    texts = [np.zeros((0, DC + 2 * DR + DC), np.uint8)] * R  # each request's rows, by what its tokens wrote
    for new in ([40, 1, 33, 0, 9, 60], [1] * 6, [1, 3, 5, 20, 1, 4], [1, 1, -1, 30, 1, 1], [2, 40, 7, 1, 1, -1], [1, 1, 1, 1, 5, 8]):
        s["new"].copy_(cuda(np.array(new, np.int32)))
        s["x"].copy_(cuda(rng.normal(size=(TOKENS, DIM)).astype(np.float32)).bfloat16())
        got = m.step(s, plan)
        assert int(s["err"]) == 0 and (plan.status == 0).all()
        start, pos = plan.token_start.cpu().numpy(), plan.start_pos.cpu().numpy()
        written = make_rows(bits_bf16(got["rows"][:, :DC]), bits_bf16(got["rows"][:, DC:]), fp8)
        few, many = np.zeros(TOKENS, bool), np.zeros(TOKENS, bool)
        first = s["row_start"].cpu().numpy()
        for r in range(R):
            a, b = start[r], start[r + 1]
            texts[r] = written[:0] if new[r] < 0 else np.concatenate([texts[r].reshape(-1, written.shape[1]) if len(texts[r]) else written[:0], written[a:b]])
            if a == b:
                assert first[r] == first[r + 1]
                continue
            assert pos[r] + b - a == len(texts[r])
            at, p = np.arange(pos[r], len(texts[r])), np.arange(len(texts[r]))
            lat, rope = row_values(texts[r], DC, fp8)
            if b - a <= FEW:
                few[a:b] = True
                assert first[r] == first[r + 1]
                for h in range(0, H, 5):
                    o, l, do, dl = attend_ref(got["qa"][a:b, h].double().cpu().numpy(), np.concatenate([lat, rope], 1), lat, at, p, m.scale, window)
                    near(s["few"][a:b, h], o, do, f"request {r} absorbed")
                    near(s["few_lse"][a:b, h], l, dl, f"request {r} absorbed lse")
            else:
                many[a:b] = True
                lo = max(0, pos[r] + 1 - window) if window else 0
                f, e = first[r], first[r + 1]
                assert e - f == len(texts[r]) - lo
                assert np.array_equal(s["latent"][f:e].double().cpu().numpy(), lat[lo:]) and np.array_equal(s["rope"][f:e].double().cpu().numpy(), rope[lo:])
                for h in range(0, H, 5):
                    kv = got["kv"][f:e, h].double().cpu().numpy()
                    o, l, do, dl = attend_ref(got["q"][a:b, h].double().cpu().numpy(), np.concatenate([kv[:, :HD], rope[lo:]], 1), kv[:, HD:], at, p[lo:], m.scale, window)
                    near(s["many"][a:b, h], o, do, f"request {r} expanded")
                    near(s["many_lse"][a:b, h], l, dl, f"request {r} expanded lse")
        for t, rest in ((s["few"], ~few), (s["few_lse"], ~few), (s["many"], ~many), (s["many_lse"], ~many)):
            assert (t.cpu()[torch.from_numpy(rest)] == 7.0).all(), "rows of other requests were written"
        s["held"].copy_(plan.seq_lens)
        s["count"].copy_(plan.free_left)


def test_both_forms_agree():
    """What the absorbed form gives for a request, through each head's values, is what the expanded form gives, but
    for roundings: of the absorbed queries (through DC products), the weights, outputs and expanded rows, each 2^-8."""
    say("[gpu] latent serving: absorbed and expanded forms of one request")
    m, rng = Layer(False, 0), np.random.default_rng(42)
    s, plan = state(rng, [FEW + 1] + [0] * (R - 1)), eg.BatchPlan(R, TOKENS)
    got = m.step(s, plan)
    absorbed = torch.zeros_like(s["few"])
    eg.engram_latent_attention(m.lay, m.pages, got["qa"], m.cache, plan, s["table"], out=absorbed)
    n = FEW + 1
    wv = m.up.view(H, 2 * HD, DC)[:, HD:].double()
    through = torch.einsum("thc,hdc->thd", absorbed[:n].double(), wv)
    # scores differ by 2^-8 of sum |q| |k| (two roundings each side), weights by that and 2^-8, values by 2^-8
    qk = got["q"][:n, :, :HD].double().abs()
    top = (qk.sum(-1).max() * got["kv"][:n, :, :HD].double().abs().max() * m.scale).item()
    d = 4 * 2.0 ** -8 * top
    bound = (torch.einsum("tc,hdc->hd", s["latent"][:n].double().abs(), wv.abs()).max().item()) * (2 * d + 4 * 2.0 ** -8)
    assert (through - s["many"][:n].double()).abs().max().item() <= bound


def test_a_captured_step_repeats_the_eager_one():
    say("[gpu] latent serving: one graph of a whole step, replayed with new tokens")
    m, rng = Layer(True, 0), np.random.default_rng(43)
    s, plan = state(rng, [20, 1, 3, 0, 9, 30]), eg.BatchPlan(R, TOKENS)
    keep = {k: s[k].clone() for k in ("table", "free")}
    m.step(s, plan)  # (before the capture: workspaces of torch's allocator)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step(s, plan)
    for k, new in enumerate(([20, 1, 3, 0, 9, 30], [1] * 6, [60, 2, 2, 2, 30, 1], [0, 0, 0, 0, 0, 0])):
        s["new"].copy_(cuda(np.array(new, np.int32)))
        s["x"].copy_(cuda(rng.normal(size=(TOKENS, DIM)).astype(np.float32)).bfloat16())
        outs = []
        for run in (graph.replay, lambda: m.step(s, plan)):
            for key, v in keep.items():
                s[key].copy_(v)
            m.cache.zero_()
            s["latent"].zero_()
            s["rope"].zero_()
            run()
            torch.cuda.synchronize()
            outs.append([s[key].clone() for key in ("few", "many", "few_lse", "many_lse", "latent", "rope", "row_start")] + [m.cache.clone()])
        for a, b in zip(*outs):
            assert torch.equal(a, b), k
    assert int(s["err"]) == 0
