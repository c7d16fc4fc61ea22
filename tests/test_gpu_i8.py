"""The 8-bit projections on the GPU against 64-bit arithmetic: quantisation is
held to the exact integers, the product to the roundings of its fp32 scaling."""
import pytest
import torch

from selective_state_space_26_b200 import (_lib, jamba_ssm_i8_proj, jamba_ssm_i8_quant,
                                           jamba_ssm_serve_get_status)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quant_ref(x):
    """scale = fp32(max|x| / 127) and q = the exact quotient rounded half to even.
    In 64 bits the quotient of an up to 24-bit x by a 24-bit scale is never taken
    for a tie that it is not: they differ by 2^-33 of it at least."""
    x = x.double()
    scale = (x.abs().amax(-1) / 127).float()
    q = torch.round(x / scale.double().unsqueeze(-1)).clamp(-127, 127)
    return torch.where(scale.unsqueeze(-1) > 0, q, 0.0), scale


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,k", [(1, 1), (3, 15), (2, 16), (5, 17), (7, 100), (64, 1024),
                                    (3, 2050), (9, 8192), (2, 20000), (130, 96)])
def test_quant_is_exact(dtype, rows, k):
    g = _gen(rows * k)
    x = (torch.randn(rows, k, generator=g, device="cuda") *
         torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)
    if k > 3:
        x[0, 1] = x[0].abs().max() / 2  # a quotient next to 63.5
        x[0, 2] = -x[0].abs().max() / 2
    q, s = jamba_ssm_i8_quant(x)
    want, scale = _quant_ref(x)
    assert q.shape == (rows, (k + 15) // 16 * 16) and torch.equal(s, scale)
    assert torch.equal(q[:, :k].double(), want)
    assert (q[:, k:] == 0).all()


def test_quant_ties_and_strides():
    """Multiples of half the scale: 127 makes the scale 1, so n + 1/2 is a tie."""
    _gen(0)
    row = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5, 0.0, -0.0, 63.5],
                       device="cuda")
    q, s = jamba_ssm_i8_quant(row[None])
    assert float(s) == 1.0
    assert q[0, :12].tolist() == [127, 0, 2, 2, 0, -2, -2, 126, -126, 0, 0, 64]
    big = torch.randn(6, 5, 70, generator=_gen(1), device="cuda").to(BF)
    for view in (big[..., 3:41], big[..., 2:50], big[:, ::1, :33], big[:2, :1, 8:24]):
        q, s = jamba_ssm_i8_quant(view)
        want, scale = _quant_ref(view)
        assert q.shape[:-1] == view.shape[:-1] and torch.equal(s, scale)
        assert torch.equal(q[..., :view.shape[-1]].double(), want)


def test_quant_of_zeros_extremes_and_non_finite():
    _gen(0)
    x = torch.zeros(7, 40, device="cuda")
    x[1, 3] = 1e-30  # a tiny row
    x[1, 4] = -0.4e-30
    x[2, 3] = 2.0 ** -140  # subnormal
    x[3, 5] = 3e38
    x[3, 6] = -1e38
    x[4, 0] = float("inf")
    x[5, 39] = float("nan")
    x[6, 7] = float("-inf")
    q, s = jamba_ssm_i8_quant(x)
    want, scale = _quant_ref(x[:4])
    assert torch.equal(s[:4], scale) and torch.equal(q[:4, :40].double(), want)
    assert torch.isnan(s[4:]).all() and (q[4:] == 0).all()
    w, ws = jamba_ssm_i8_quant(torch.randn(5, 40, generator=_gen(2), device="cuda"))
    out = jamba_ssm_i8_proj(q, s, w, ws, out_dtype=F32)
    assert (out[0] == 0).all() and torch.isnan(out[4:]).all()
    # huge and tiny scales: what fp32 can hold comes out, whatever acc * scale alone would do
    v, e = _proj_ref(q[:4], s[:4], w, ws, None, F32)
    top = torch.finfo(F32).max
    assert torch.equal(torch.isinf(out[:4]), v.abs() > top)
    held = v.abs() <= top
    # a subnormal product is rounded to a multiple of 2^-149
    assert ((out[:4].double() - v).abs()[held] <= e[held] + 2.0 ** -149).all()
    assert held[3].any()


def _proj_ref(q, s, w, ws, bias, dtype):
    """(value, bound): the sum is exact, its conversion, the two products and the
    bias round once each (2^-24 of the value at that point), then the output."""
    acc = q.double() @ w.double().T
    v = acc * s.double()[..., None] * ws.double()
    e = 3 * 2.0 ** -24 * v.abs()
    if bias is not None:
        v = v + bias.double()
        e = e + 2.0 ** -24 * v.abs()
    return v, e * 1.01 + (2.0 ** -8 if dtype == BF else 0.0) * (v.abs() + e)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,k,n", [
    (1, 1, 1), (1, 16, 8), (2, 130, 100), (8, 512, 256), (16, 1000, 77), (17, 128, 129),
    (33, 4096, 300), (64, 96, 1024), (100, 2050, 257), (128, 128, 128), (129, 144, 130),
    (200, 640, 513), (257, 1040, 255), (300, 2048, 1030), (1000, 272, 96), (515, 8208, 384),
])
def test_proj_matches(dtype, m, k, n):
    g = _gen(m + 3 * k + 7 * n)
    pitch = (k + 15) // 16 * 16
    q = torch.zeros(m, pitch, dtype=torch.int8, device="cuda")
    w = torch.zeros(n, pitch, dtype=torch.int8, device="cuda")
    q[:, :k] = torch.randint(-128, 128, (m, k), generator=g, device="cuda").to(torch.int8)
    w[:, :k] = torch.randint(-128, 128, (n, k), generator=g, device="cuda").to(torch.int8)
    s = torch.rand(m, generator=g, device="cuda") + 0.1
    ws = torch.rand(n, generator=g, device="cuda") + 0.1
    for bias in (None, torch.randn(n, generator=g, device="cuda") * 100):
        buf = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
        out = jamba_ssm_i8_proj(q, s, w, ws, bias=bias, out=buf[:m])
        v, e = _proj_ref(q, s, w, ws, bias, dtype)
        over = (out.double() - v).abs() - e
        assert float(over.max()) <= 0, (float(over.max()), int(over.argmax()))
        assert (buf[m] == 7).all(), "a row behind the last was written"
    assert jamba_ssm_serve_get_status() == 0


def test_proj_extreme_sums():
    """-128 * -128 * K at the largest K reaches 2^31 - 2^18: the sum must not wrap."""
    _gen(0)
    k = _lib.I8_MAX_K
    q = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, k), -128, dtype=torch.int8, device="cuda")
    q[1], w[3] = 127, 127
    one = torch.ones(5, device="cuda")
    out = jamba_ssm_i8_proj(q, one[:3], w, one, out_dtype=F32)
    v, e = _proj_ref(q, one[:3], w, one, None, F32)
    assert ((out.double() - v).abs() <= e).all()


def test_proj_empty_leading_shapes_and_out():
    g = _gen(5)
    x = torch.randn(2, 3, 50, generator=g, device="cuda").to(BF)
    w, ws = jamba_ssm_i8_quant(torch.randn(20, 50, generator=g, device="cuda"))
    q, s = jamba_ssm_i8_quant(x)
    assert q.shape == (2, 3, 64) and s.shape == (2, 3)
    out = jamba_ssm_i8_proj(q, s, w, ws)
    assert out.shape == (2, 3, 20) and out.dtype == BF
    flat = jamba_ssm_i8_proj(q.view(6, 64), s.view(6), w, ws)
    assert torch.equal(out.view(6, 20), flat)
    q1, s1 = jamba_ssm_i8_quant(x[1, 2])  # one row, without leading dimensions
    assert q1.shape == (64,) and s1.shape == ()
    one = jamba_ssm_i8_proj(q1, s1, w, ws)
    assert one.shape == (20,) and torch.equal(one, out[1, 2])
    q0, s0 = jamba_ssm_i8_quant(x[:0])
    assert jamba_ssm_i8_proj(q0, s0, w, ws).shape == (0, 3, 20)


def test_quantised_linear_is_near_the_float_one():
    """x W^T itself: q is off by half a step, so an output by at most
    sum_k (|x| s_w/2 + |w| s_x/2 + s_x s_w/4)."""
    g = _gen(8)
    x = torch.randn(40, 700, generator=g, device="cuda")
    w = torch.randn(90, 700, generator=g, device="cuda")
    q, s = jamba_ssm_i8_quant(x)
    wq, ws = jamba_ssm_i8_quant(w)
    out = jamba_ssm_i8_proj(q, s, wq, ws, out_dtype=F32).double()
    xd, wd, sd, wsd = x.double(), w.double(), s.double()[:, None], ws.double()
    bound = xd.abs().sum(1, keepdim=True) * wsd / 2 + wd.abs().sum(1) * sd / 2 + 700 * sd * wsd / 4
    assert ((out - xd @ wd.T).abs() <= bound * (1 + 1e-5)).all()


@pytest.mark.parametrize("k,n", [(64, 2048), (1000, 1027), (4096, 512)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_tokens_do_not_depend_on_their_batch(k, n, dtype):
    """Other token counts take other tiles and other splits of K; the sums are of
    integers and the scales' order is fixed, so every bit stays."""
    g = _gen(12)
    m = 2305
    q, s = jamba_ssm_i8_quant(torch.randn(m, k, generator=g, device="cuda"))
    w, ws = jamba_ssm_i8_quant(torch.randn(n, k, generator=g, device="cuda"))
    # scales of every size, some outside of what the fast order of the factors takes
    s[::7] *= 2.0 ** 62
    s[3::11] *= 2.0 ** -70
    s[5::13] = 0.0
    ws[::5] *= 2.0 ** -64
    bias = torch.randn(n, generator=g, device="cuda")
    out = jamba_ssm_i8_proj(q, s, w, ws, bias=bias, out_dtype=dtype)
    for a, b in [(0, 1), (2304, 2305), (255, 272), (17, 49), (1000, 1064), (250, 450), (5, 905)]:
        assert torch.equal(out[a:b], jamba_ssm_i8_proj(q[a:b], s[a:b], w, ws, bias=bias,
                                                       out_dtype=dtype)), (a, b)


def test_offsets_past_32_bits():
    """2.2e9 inputs and outputs: the last rows are those of the same tokens alone."""
    g = _gen(11)
    m, k, n = 140_000, 15_984, 16_000
    x = torch.randn(m, k, generator=g, device="cuda", dtype=BF)
    q, s = jamba_ssm_i8_quant(x)
    qt, st = jamba_ssm_i8_quant(x[-300:])
    assert torch.equal(q[-300:], qt) and torch.equal(s[-300:], st)
    del x
    w, ws = jamba_ssm_i8_quant(torch.randn(n, 64, generator=g, device="cuda"))
    thin = q[:, :64].contiguous()
    out = jamba_ssm_i8_proj(thin, s, w, ws)
    assert torch.equal(out[-300:], jamba_ssm_i8_proj(thin[-300:], s[-300:], w, ws))
    assert torch.equal(out[:300], jamba_ssm_i8_proj(thin[:300], s[:300], w, ws))
    assert jamba_ssm_serve_get_status() == 0


def test_graph_and_streams():
    g = _gen(9)
    x = torch.randn(300, 1000, generator=g, device="cuda").to(BF)
    w, ws = jamba_ssm_i8_quant(torch.randn(500, 1000, generator=g, device="cuda"))
    step = lambda v: jamba_ssm_i8_proj(*jamba_ssm_i8_quant(v), w, ws)  # noqa: E731
    static = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(static)
    static.copy_(x.flip(0))
    want_new, want_old = step(x.flip(0).contiguous()), step(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        eager = step(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, want_new) and torch.equal(eager, want_old)
    q, s = jamba_ssm_i8_quant(x, stream=side)
    out = jamba_ssm_i8_proj(q, s, w, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want_old)


@pytest.mark.parametrize("m,k,n", [(8, 1024, 256), (8, 4096, 300), (100, 256, 128), (900, 2048, 4096)])
def test_waits_that_run_out_are_reported(m, k, n):
    """The first copies withheld: the kernel gives its waits up, records the
    timeout and ends; the next call is whole again."""
    g = _gen(3)
    q, s = jamba_ssm_i8_quant(torch.randn(m, k, generator=g, device="cuda"))
    w, ws = jamba_ssm_i8_quant(torch.randn(n, k, generator=g, device="cuda"))
    good = jamba_ssm_i8_proj(q, s, w, ws)
    assert jamba_ssm_serve_get_status() == 0
    jamba_ssm_i8_proj(q, s, w, ws, timeout_cycles=2_000_000, debug_flags=1)
    assert jamba_ssm_serve_get_status() == _lib.ERR_TIMEOUT
    assert torch.equal(jamba_ssm_i8_proj(q, s, w, ws), good)
    assert jamba_ssm_serve_get_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,k,n", [(8, 8192, 4096), (3, 4096, 300), (64, 8192, 1024)])
def test_no_part_of_a_sum_is_written(m, k, n, dtype):
    """One of the CTAs that share a tile's K gives its waits up: the others, whose
    copies all arrived, write nothing of that tile either."""
    g = _gen(4)
    q, s = jamba_ssm_i8_quant(torch.randn(m, k, generator=g, device="cuda"))
    w, ws = jamba_ssm_i8_quant(torch.randn(n, k, generator=g, device="cuda"))
    good = jamba_ssm_i8_proj(q, s, w, ws, out_dtype=dtype)
    out = torch.full_like(good, 12345.0)
    jamba_ssm_i8_proj(q, s, w, ws, out=out, timeout_cycles=2_000_000, debug_flags=2)
    assert jamba_ssm_serve_get_status() == _lib.ERR_TIMEOUT
    assert ((out == torch.full_like(out, 12345.0)) | (out == good)).all()
    assert not torch.equal(out, good)
    assert torch.equal(jamba_ssm_i8_proj(q, s, w, ws, out_dtype=dtype), good)
    assert jamba_ssm_serve_get_status() == 0


def test_refusals():
    g = _gen(1)
    q, s = jamba_ssm_i8_quant(torch.randn(4, 32, generator=g, device="cuda"))
    w, ws = jamba_ssm_i8_quant(torch.randn(6, 32, generator=g, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        jamba_ssm_i8_quant(torch.randn(4, 32))
    with pytest.raises(TypeError):
        jamba_ssm_i8_quant(torch.randn(4, 32, device="cuda").half())
    with pytest.raises(ValueError, match="rows"):
        jamba_ssm_i8_quant(torch.randn(32, 4, device="cuda").T)
    with pytest.raises(ValueError, match="multiple of 16"):
        jamba_ssm_i8_proj(q[:, :20].contiguous(), s, w, ws)
    with pytest.raises(ValueError, match="contiguous"):
        jamba_ssm_i8_proj(q[:, :16], s, w[:, :16].contiguous(), ws)
    with pytest.raises(ValueError, match="shape"):
        jamba_ssm_i8_proj(q, s, w[:, :16].contiguous(), ws)
    with pytest.raises(ValueError, match="shape"):
        jamba_ssm_i8_proj(q, s[:3], w, ws)
    with pytest.raises(TypeError):
        jamba_ssm_i8_proj(q, s.double(), w, ws)
    with pytest.raises(TypeError):
        jamba_ssm_i8_proj(q, s, w, ws, out_dtype=torch.float16)
    with pytest.raises(_lib.JambaSSMError):
        jamba_ssm_i8_quant(torch.randn(4, 0, device="cuda"))
