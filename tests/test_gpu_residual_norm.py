"""engram_residual_norm against its formula in 64 bits (the bounds are derived in serving_common.norm_ref):
types, gates, shared and strided block outputs, closed tokens, odd and large rows, and in-place calls."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from serving_common import near, norm_ref  # noqa: E402

GATES = ("none", "token", "feature")


def inputs(M, hc, dim, ys, fp32, gate, seed=0, strided=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0, std, generator=g)
    x = normal(1, M, hc, dim)
    x[:, ::7] *= 50
    d = dict(x=x if fp32 else x.bfloat16(), gate=None)
    d["y"] = normal(1, M, (ys + 2) * dim).bfloat16()[..., 2 * dim:].view(1, M, ys, dim) if strided else \
        normal(1, M, ys, dim).bfloat16()
    if gate == "token":
        d["gate"] = torch.rand((1, M, hc), device="cuda", generator=g)
    elif gate == "feature":
        d["gate"] = normal(1, M, 3 * ys * dim, std=3).bfloat16()[..., ys * dim:2 * ys * dim].view(1, M, ys, dim) if strided \
            else normal(1, M, ys, dim, std=3).bfloat16()
    d["post_weight"], d["pre_weight"] = 1 + 0.3 * normal(hc, dim), 1 + 0.3 * normal(hc, dim)
    d["token_mask"] = (torch.rand((1, M), device="cuda", generator=g) > 0.2).to(torch.uint8)
    return d


def lay(hc, dim, ys, fp32, gate, **kw):
    kw = dict(alpha=0.9, beta=-1.3, post_eps=1e-6, pre_eps=1e-5) | kw
    return eg.make_norm_layout(hc, dim, y_streams=ys, gate=GATES.index(gate),
                               stream_format=eg.STREAM_FP32 if fp32 else eg.STREAM_BF16, **kw)


def check(l, d, gate, **kw):
    out, h = eg.engram_residual_norm(l, d["x"], d["y"], gate=d["gate"], post_weight=d["post_weight"],
                                     pre_weight=d["pre_weight"], token_mask=d["token_mask"], **kw)
    r, hr, br, bh = norm_ref(d["x"], d["y"], d["gate"], gate, d["post_weight"], d["pre_weight"], d["token_mask"], l.alpha, l.beta,
                             l.post_eps, l.pre_eps, bool(l.post_norm))
    near(out, r, br, "out")
    if l.pre_norm:
        near(h, hr, bh, "h")
    if d["token_mask"] is not None:
        shut = ~d["token_mask"].bool()
        assert torch.equal(out[shut], d["x"][shut])
    return out, h


@pytest.mark.parametrize("dim", [8, 64, 72, 512, 520, 1000, 1024, 2056, 4096, 5120, 5128, 8192, 10240, 16384, 20008, 32768,
                                 40960])
@pytest.mark.parametrize("fp32", [False, True])
def test_row_lengths(dim, fp32):
    say(f"[gpu] residual norm: dim {dim}, {'fp32' if fp32 else 'bf16'} streams")
    for hc, M in ((1, 5), (4, 3)):
        check(lay(hc, dim, hc, fp32, "token"), inputs(M, hc, dim, hc, fp32, "token", seed=dim), "token")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("ys,hc", [(1, 1), (1, 4), (4, 4), (1, 3), (3, 3), (1, 64)])
@pytest.mark.parametrize("post", [True, False])
def test_gates_and_shared_outputs(gate, ys, hc, post):
    say(f"[gpu] residual norm: gate {gate}, {ys} of {hc} streams, post norm {post}")
    for fp32 in (False, True):
        for strided in (False, True):
            for M in (1, 2, 33):
                check(lay(hc, 136, ys, fp32, gate, post_norm=post), inputs(M, hc, 136, ys, fp32, gate, seed=M, strided=strided),
                      gate)


def test_value_slice_of_a_projection_row():
    say("[gpu] residual norm: y is the value slice of kv rows, gate from engram_gate_apply's shape")
    M, dim = 70, 5120
    d = inputs(M, 4, dim, 1, False, "token", seed=9)
    kv = torch.randn((1, M, 5 * dim), device="cuda").bfloat16()
    d["y"] = kv[..., 4 * dim:].view(1, M, 1, dim)
    check(lay(4, dim, 1, False, "token"), d, "token")


@pytest.mark.parametrize("fp32", [False, True])
def test_parts_alone_and_in_place(fp32):
    say(f"[gpu] residual norm: without a block, without the next norm, without weights or mask, in place ({fp32})")
    d = inputs(37, 2, 320, 2, fp32, "none", seed=4)
    l = lay(2, 320, 2, fp32, "none")
    x, h = eg.engram_residual_norm(l, d["x"], pre_weight=d["pre_weight"])
    assert x is d["x"]
    _, hr, _, bh = norm_ref(d["x"], None, None, "none", None, d["pre_weight"], None, 1, 1, 0, l.pre_eps)
    near(h, hr, bh, "h alone")
    only = lay(2, 320, 2, fp32, "none", pre_norm=False)
    out, none = check(only, d, "none")
    assert none is None
    for k in ("post_weight", "pre_weight", "token_mask"):
        check(l, dict(d, **{k: None}), "none")
    ref, h_ref = check(l, d, "none")
    y = d["x"].clone()
    got, h = eg.engram_residual_norm(l, y, d["y"], post_weight=d["post_weight"], pre_weight=d["pre_weight"],
                                     token_mask=d["token_mask"].bool(), out=y)
    assert got is y and torch.equal(y, ref) and torch.equal(h, h_ref)


def test_closed_tokens_hide_what_they_hold():
    say("[gpu] residual norm: NaN and infinities in closed tokens' y and gate; all closed")
    for gate in ("token", "feature"):
        d = inputs(20, 2, 264, 1, False, gate, seed=2)
        ref, h_ref = check(lay(2, 264, 1, False, gate), d, gate)
        shut = ~d["token_mask"].bool()
        d["y"][shut] = float("nan")
        d["gate"][shut] = float("inf")
        out, h = eg.engram_residual_norm(lay(2, 264, 1, False, gate), d["x"], d["y"], gate=d["gate"],
                                         post_weight=d["post_weight"], pre_weight=d["pre_weight"],
                                         token_mask=d["token_mask"])
        assert torch.equal(out, ref) and torch.equal(h, h_ref)
        out, _ = eg.engram_residual_norm(lay(2, 264, 1, False, gate), d["x"], d["y"], gate=d["gate"],
                                         token_mask=torch.zeros_like(d["token_mask"]))
        assert torch.equal(out, d["x"])


def test_zero_rows_and_large_values():
    say("[gpu] residual norm: rows of zeros, values near the largest")
    d = inputs(6, 1, 128, 1, True, "none", seed=6)
    d["y"][:, 0] = 0
    d["x"][:, 0] = 0
    d["y"][:, 1] = 1e18
    d["x"][:, 2] = 1e-19
    d["token_mask"] = None
    check(lay(1, 128, 1, True, "none"), d, "none")
    check(lay(1, 128, 1, True, "none", post_eps=1e-20, pre_eps=1e-20), d, "none")


def test_rows_past_32_bit_offsets():
    say("[gpu] residual norm: a strided y past 2^32 bytes")
    M, dim = 9, 64
    stride = 1 << 28  # 2^28 elements, 512 MiB between tokens
    buf = torch.zeros(stride * (M - 1) + dim, dtype=torch.bfloat16, device="cuda")
    y = buf.as_strided((1, M, 1, dim), (stride * M, stride, dim, 1))
    y.copy_(torch.randn((1, M, 1, dim), device="cuda"))
    d = inputs(M, 1, dim, 1, False, "none", seed=8)
    d["y"] = y
    check(lay(1, dim, 1, False, "none"), d, "none")


def test_captured_and_replayed():
    say("[gpu] residual norm: a captured call, replayed between eager work")
    d = inputs(50, 4, 640, 1, False, "token", seed=3)
    l = lay(4, 640, 1, False, "token")
    args = dict(gate=d["gate"], post_weight=d["post_weight"], pre_weight=d["pre_weight"], token_mask=d["token_mask"])
    out, h = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    eg.engram_residual_norm(l, d["x"], d["y"], out=out, h=h, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.engram_residual_norm(l, d["x"], d["y"], out=out, h=h, **args)
    for k in range(3):
        d["x"].mul_(1.5)
        ref, h_ref = eg.engram_residual_norm(l, d["x"], d["y"], **args)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(h, h_ref), k


@pytest.mark.parametrize("fp32", [False, True])
def test_closed_tokens_keep_their_bits(fp32):
    say(f"[gpu] residual norm: every bit pattern of a closed token, {'fp32' if fp32 else 'bf16'}")
    bits = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32)
    x = ((bits << 16) | (bits & 0x7FFF)).view(torch.float32) if fp32 else bits.to(torch.int16).view(torch.bfloat16)
    x = x.view(1, 64, 1, 1024)
    mask = torch.zeros((1, 64), dtype=torch.uint8, device="cuda")
    y = torch.full_like(x, float("nan"), dtype=torch.bfloat16)
    out, _ = eg.engram_residual_norm(lay(1, 1024, 1, fp32, "none"), x, y, token_mask=mask)
    as_int = torch.int32 if fp32 else torch.int16
    assert torch.equal(out.view(as_int), x.view(as_int))
