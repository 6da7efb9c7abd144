"""engram_linear: exact on small whole numbers (every product and sum fits fp32, so any wrong index shows),
and within the derived bound (serving_common.linear_ref) on random values; odd sizes, strides, activations,
the gated form, residuals in place, single tokens."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from serving_common import linear_ref, near  # noqa: E402

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")


def lay(K, N, act="none", glu=False, fp32=False):
    return eg.make_linear_layout(K, N, activation=ACTS.index(act), glu=glu,
                                 stream_format=eg.STREAM_FP32 if fp32 else eg.STREAM_BF16)


def whole(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").float()


SIZES = [(1, 64, 16), (1, 8, 1), (1, 5120, 5120), (2, 72, 33), (5, 1000, 257), (16, 128, 64), (17, 640, 100), (31, 4096, 48),
         (33, 200, 1001), (64, 1024, 512), (65, 264, 130), (100, 5120, 1030), (127, 64, 255), (128, 4096, 256), (129, 520, 384),
         (200, 2048, 1280), (257, 1288, 513), (300, 8, 700), (512, 512, 2048), (777, 1032, 777), (1025, 256, 1281),
         (8, 4104, 47), (13, 3000, 130), (16, 4104, 47), (9, 264, 9001), (3, 56, 20000), (7, 192, 20001)]


# shapes that take every tile, whole and split over K (plain, then gated), as engram_linear chooses them on
# 256 compute units; odd on purpose in tokens, features and the rest of K past whole stages
TILES = [(2067, 256, 4991), (1803, 832, 3400), (822, 4912, 3006), (512, 4560, 5198), (1537, 312, 3597), (136, 5144, 3845),
         (1678, 120, 2371), (1887, 5352, 260), (822, 280, 5993), (161, 3840, 5879), (385, 64, 4707), (65, 4816, 5955),
         (1043, 64, 3868), (1594, 64, 2501), (163, 3536, 5707), (229, 416, 4108), (35, 4008, 5463), (202, 64, 4108),
         (68, 3168, 2882), (2048, 4096, 4096), (1000, 10240, 5120), (681, 3744, 36), (166, 2936, 5874), (267, 3480, 3808)]
GATED_TILES = [(963, 248, 4830), (1561, 840, 1828), (331, 4936, 2714), (1163, 1032, 3214), (194, 4736, 4267), (391, 120, 4618),
               (146, 4336, 1833), (323, 280, 5664), (66, 4072, 5545), (925, 304, 3182), (173, 4016, 2770), (67, 4688, 2727),
               (385, 64, 4707), (258, 64, 5478), (180, 3296, 2738), (33, 2936, 4279), (71, 64, 4218), (73, 3392, 1381),
               (691, 3888, 17), (301, 5120, 10240), (936, 240, 5235), (484, 832, 5870),
               (222, 4424, 5244), (215, 4640, 5264), (136, 5136, 1831), (2038, 5552, 1544),
               (69, 4152, 2767), (162, 2832, 2780), (1369, 3008, 17), (17, 2232, 260), (263, 3416, 1890)]


@pytest.mark.parametrize("M,K,N,glus", [(*s, (False, True)) for s in SIZES] + [(*s, (False,)) for s in TILES] +
                         [(*s, (True,)) for s in GATED_TILES])
def test_exact_on_whole_numbers(M, K, N, glus):
    say(f"[gpu] linear: {M} x {K} x {N}, whole numbers")
    g = torch.Generator(device="cuda").manual_seed(M * 7 + N)
    for glu in glus:
        rows = 2 * N if glu else N
        x, w, b, r = whole(g, M, K), whole(g, rows, K), whole(g, rows), whole(g, M, N)
        # |z| <= 9 K + 3 < 2^17; gated products are kept below 2^24 by a sparse weight
        if glu:
            w = w * (torch.rand((rows, K), generator=g, device="cuda") < min(1.0, 64 / K))
        z = x.double() @ w.double().T + b.double()
        ref = (z[:, :N] * z[:, N:] if glu else z) + r.double()
        assert ref.abs().max() < 2 ** 24
        got = eg.engram_linear(lay(K, N, glu=glu, fp32=True), x.bfloat16(), w.bfloat16(), bias=b, residual=r)
        assert torch.equal(got.double(), ref), (glu, (got.double() != ref).nonzero()[:4].tolist())
        got = eg.engram_linear(lay(K, N, glu=glu), x.bfloat16(), w.bfloat16())
        z = x.double() @ w.double().T
        ref = (z[:, :N] * z[:, N:] if glu else z).float().bfloat16()
        assert torch.equal(got, ref), glu


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("glu", [False, True])
def test_activations(act, glu):
    say(f"[gpu] linear: {act}, gated {glu}")
    g = torch.Generator(device="cuda").manual_seed(11)
    for M, K, N in ((1, 256, 96), (40, 520, 130), (150, 384, 264)):
        rows = 2 * N if glu else N
        x = torch.empty((M, K), device="cuda").normal_(generator=g).bfloat16()
        w = torch.empty((rows, K), device="cuda").normal_(0, 3 * K ** -0.5, generator=g).bfloat16()
        b = torch.empty(rows, device="cuda").normal_(generator=g)
        for fp32 in (False, True):
            dt = torch.float32 if fp32 else torch.bfloat16
            r = torch.empty((M, N), device="cuda").normal_(generator=g).to(dt)
            for bias, res in ((None, None), (b, None), (None, r), (b, r)):
                got = eg.engram_linear(lay(K, N, act, glu, fp32), x, w, bias=bias, residual=res)
                assert got.dtype == dt
                near(got, *linear_ref(x, w, bias, res, act, glu, dt), f"{M} {fp32}")


def test_saturated_activations_stay_finite():
    say("[gpu] linear: activations of very large arguments")
    x = torch.full((3, 64), 100.0, device="cuda").bfloat16()
    w = torch.cat([torch.full((8, 64), 50.0), torch.full((8, 64), -50.0)]).cuda().bfloat16()
    for act, hi, lo in (("relu", 3.2e5, 0), ("gelu", 3.2e5, 0), ("gelu_tanh", 3.2e5, 0), ("silu", 3.2e5, 0), ("sigmoid", 1, 0)):
        got = eg.engram_linear(lay(64, 16, act, fp32=True), x, w)
        assert torch.equal(got[:, :8], torch.full_like(got[:, :8], hi)) and (got[:, 8:] == lo).all(), act


@pytest.mark.parametrize("M", [1, 30, 90, 200])
def test_slices_and_in_place(M):
    say(f"[gpu] linear: slices of wider rows, leading dimensions, the residual in place, {M} tokens")
    g = torch.Generator(device="cuda").manual_seed(M)
    K, N = 328, 200
    wide = whole(g, M, 3 * K).bfloat16()
    x, w = wide[:, K:2 * K], whole(g, N, K).bfloat16()
    for fp32 in (False, True):
        dt = torch.float32 if fp32 else torch.bfloat16
        for pad in (8, 3):
            buf = torch.full((M, N + pad), 5.0, device="cuda", dtype=dt)
            res = whole(g, M, N + 16).to(dt)[:, :N]
            z = x.double() @ w.double().T
            got = eg.engram_linear(lay(K, N, fp32=fp32), x, w, residual=res, out=buf[:, :N])
            ref = (z + res.double()).float().to(dt)
            assert got.data_ptr() == buf.data_ptr() and torch.equal(buf[:, :N], ref)
            assert (buf[:, N:] == 5).all()
            stream = res.clone()
            again = eg.engram_linear(lay(K, N, fp32=fp32), x, w, residual=stream, out=stream)
            assert again is stream and torch.equal(stream, ref)
    if M % 2 == 0:
        y = eg.engram_linear(lay(K, N), x.view(2, M // 2, K) if x.is_contiguous() else x.unflatten(0, (2, M // 2)), w)
        assert y.shape == (2, M // 2, N) and torch.equal(y.reshape(M, N), eg.engram_linear(lay(K, N), x, w))


def test_what_lies_behind_the_rows_is_not_read():
    say("[gpu] linear: NaN behind the last feature of x and behind its last row")
    g = torch.Generator(device="cuda").manual_seed(1)
    for M, K, N in ((1, 72, 40), (20, 200, 90), (70, 136, 130), (190, 72, 260)):
        buf = torch.full((M + 3, K + 56), float("nan"), device="cuda").bfloat16()
        buf[:M, :K] = whole(g, M, K).bfloat16()
        wbuf = torch.full((N + 5, K), float("nan"), device="cuda").bfloat16()
        wbuf[:N] = whole(g, N, K).bfloat16()
        out = torch.full((M + 2, N), 9.0, device="cuda")
        eg.engram_linear(lay(K, N, fp32=True), buf[:M, :K], wbuf[:N], out=out[:M])
        assert torch.equal(out[:M].double(), buf[:M, :K].double() @ wbuf[:N].double().T)
        assert (out[M:] == 9).all()


def test_infinities_and_nan_stay_in_their_rows():
    say("[gpu] linear: an infinity and a NaN in one token, one in one weight row")
    g = torch.Generator(device="cuda").manual_seed(1)
    for M in (8, 80, 200):
        x, w = whole(g, M, 128).bfloat16(), whole(g, 140, 128).bfloat16()
        ref = eg.engram_linear(lay(128, 140, fp32=True), x, w)
        x2, w2 = x.clone(), w.clone()
        x2[5, 3] = float("nan")
        w2[77, 9] = float("inf")
        got = eg.engram_linear(lay(128, 140, fp32=True), x2, w2)
        keep = torch.ones_like(ref, dtype=torch.bool)
        keep[5], keep[:, 77] = False, False
        assert torch.equal(got[keep], ref[keep])
        assert got[5].isnan().all() and not got[x[:, 9].float().ne(0), 77].isfinite().any()


def test_rows_past_32_bit_offsets():
    say("[gpu] linear: x and out rows past 2^32 bytes")
    g = torch.Generator(device="cuda").manual_seed(2)
    M, K, N, far = 20, 64, 48, 1 << 27
    xb = torch.zeros(far * (M - 1) + K, dtype=torch.bfloat16, device="cuda")
    ob = torch.zeros(far * (M - 1) + N, dtype=torch.bfloat16, device="cuda")
    x, out = xb.as_strided((M, K), (far, 1)), ob.as_strided((M, N), (far, 1))
    x.copy_(whole(g, M, K))
    w = whole(g, N, K).bfloat16()
    eg.engram_linear(lay(K, N), x, w, out=out)
    assert torch.equal(out, (x.double() @ w.double().T).float().bfloat16())


def test_on_a_side_stream_and_captured():
    say("[gpu] linear: another stream, and a captured call replayed between eager work")
    g = torch.Generator(device="cuda").manual_seed(4)
    for M in (4, 60, 300):
        x, w = whole(g, M, 512).bfloat16(), whole(g, 640, 512).bfloat16()
        l, out = lay(512, 640, "relu"), torch.empty((M, 640), dtype=torch.bfloat16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            eg.engram_linear(l, x, w, out=out)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, eg.engram_linear(l, x, w))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eg.engram_linear(l, x, w, out=out)
        for k in range(3):
            x.neg_()
            ref = eg.engram_linear(l, x, w)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref), (M, k)


def test_workspace_is_checked_and_kept_to():
    say("[gpu] linear: a caller's workspace, one that is too small, bytes around it")
    g = torch.Generator(device="cuda").manual_seed(5)
    M, K, N = 100, 5120, 1030
    l = lay(K, N, fp32=True)
    need = eg.engram_linear_workspace_bytes(l, M)
    assert need > 0 and eg.engram_linear_workspace_bytes(lay(64, 64), 4) == 0
    x, w = whole(g, M, K).bfloat16(), whole(g, N, K).bfloat16()
    ref = x.double() @ w.double().T
    buf = torch.full((need + 512,), 171, dtype=torch.uint8, device="cuda")
    got = eg.engram_linear(l, x, w, workspace=buf[256:256 + need])
    assert torch.equal(got.double(), ref) and (buf[:256] == 171).all() and (buf[256 + need:] == 171).all()
    out = torch.full((M, N), 3.0, device="cuda")
    for bad in (buf[:need - 16], buf[8:8 + need]):
        with pytest.raises(eg.EngramError) as e:
            eg.engram_linear(l, x, w, out=out, workspace=bad)
        assert e.value.status == -5
    torch.cuda.synchronize()
    assert (out == 3).all()


def test_split_calls_at_the_same_time():
    say("[gpu] linear: split calls on two streams, and two captured graphs replayed together")
    g = torch.Generator(device="cuda").manual_seed(6)
    M, K, N = 100, 5120, 1030
    l = lay(K, N, fp32=True)
    assert eg.engram_linear_workspace_bytes(l, M) > 0
    xs = [whole(g, M, K).bfloat16() for _ in range(2)]
    w = whole(g, N, K).bfloat16()
    refs = [x.double() @ w.double().T for x in xs]
    outs = [torch.empty((M, N), device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, o, s in zip(xs, outs, streams):
            with torch.cuda.stream(s):
                eg.engram_linear(l, x, w, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o.double(), r) for o, r in zip(outs, refs))
    graphs = []
    for x, o in zip(xs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            eg.engram_linear(l, x, w, out=o)
    for k in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for gr, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o.double(), r) for o, r in zip(outs, refs)), k
