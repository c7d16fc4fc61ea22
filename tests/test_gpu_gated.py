"""The gated linear recurrence on the GPU against the 64-bit recurrence, within
the bounds that tests/gated_ref.py derives: whole sequences, packed ones, state
slots, the backward pass, the one-token update, and what each refuses."""
import pytest
import torch

from selective_state_space_26_b200 import (_lib, jamba_ssm_gated_get_status, jamba_ssm_gated_scan,
                                           jamba_ssm_gated_scan_bwd, jamba_ssm_gated_scan_ckpt,
                                           jamba_ssm_gated_scan_ckpt_size,
                                           jamba_ssm_gated_state_update)
from tests.gated_ref import Reference, assert_within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


def _inputs(shape, dtype, seed, gate=True, strided=False, slow=False):
    """x, g, z (or None), rate, bias; strided: column blocks of one buffer."""
    dev, d = _dev(), shape[-1]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    if strided:
        buf = r(*shape[:-1], 3 * d + 2).to(dtype)
        x, g, z = buf[..., :d], buf[..., d:2 * d], buf[..., 2 * d:3 * d]
    else:
        x, g, z = (r(*shape).to(dtype) for _ in range(3))
    rate = torch.rand(d, generator=gen, device=dev) ** (8 if slow else 1)
    return x, g, z if gate else None, rate, r(d)


def _check_scan(ref, out, hf, what):
    assert_within(out, ref.out, ref.e_out, f"{what}: out")
    if hf is not None:
        assert_within(hf, ref.h_final, ref.e_final, f"{what}: h_final")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,seqlen,d", [
    (1, 1, 1), (2, 1, 64), (1, 7, 3), (3, 63, 33), (1, 64, 128), (2, 65, 62), (1, 200, 96),
    (2, 513, 130), (1, 1100, 24), (5, 129, 257), (1, 4099, 16),
])
def test_scan_matches_recurrence(dtype, batch, seqlen, d):
    x, g, z, rate, bias = _inputs((batch, seqlen, d), dtype, 7 * d + seqlen, slow=seqlen > 300)
    h0 = torch.randn(batch, d, device=x.device)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0)
    _check_scan(Reference(x, g, z, rate, bias, h0), out, hf, f"{batch}x{seqlen}x{d}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,seqlen,d", [(40, 150, 512), (24, 300, 320), (24, 150, 310),
                                             (2, 700, 2048)])
def test_scan_of_many_tiles(dtype, batch, seqlen, d):
    """Enough channel tiles for the whole device: the cuts without clusters."""
    x, g, z, rate, bias = _inputs((batch, seqlen, d), dtype, d)
    h0 = torch.randn(batch, d, device=x.device)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0)
    _check_scan(Reference(x, g, z, rate, bias, h0), out, hf, f"{batch}x{seqlen}x{d}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_whose_product_leaves_the_range(dtype):
    """Neighbouring channels closed to e^-50 each: their exponentials' product is
    past fp32, and the small rates must come out as they are, not as 0."""
    x, g, z, rate, bias = _inputs((1, 200, 64), dtype, 2)
    g[:] = -50.0
    z[:, :, ::2] = -60.0
    rate[:] = 1.0
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate)
    ref = Reference(x, g, z, rate)
    _check_scan(ref, out, hf, "closed pairs")
    assert (hf != 0).all()
    rel = (hf.double().cpu() - ref.h_final).norm() / ref.h_final.norm()
    assert rel < 200 * 2.0 ** -22  # each rate is within (50 + 8) 2^-23, each sum 2^-24


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_optional_arguments(dtype):
    x, g, z, rate, bias = _inputs((2, 100, 40), dtype, 3)
    out, hf = jamba_ssm_gated_scan(x, g)
    _check_scan(Reference(x, g), out, hf, "bare")
    out, hf = jamba_ssm_gated_scan(x, g, z=z, return_final_state=False)
    assert hf is None
    _check_scan(Reference(x, g, z), out, None, "gate only")
    out, hf = jamba_ssm_gated_scan(x, g, rate=rate)
    _check_scan(Reference(x, g, rate=rate), out, hf, "rate only")
    buf = torch.empty_like(x)
    h = torch.randn(2, 40, device=x.device)
    ref = Reference(x, g, bias=bias, h0=h)
    out, hf = jamba_ssm_gated_scan(x, g, bias=bias, h0=h, h_final=h, out=buf)  # in place
    assert out is buf and hf is h
    _check_scan(ref, out, hf, "state in place")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 63, 200])
def test_strided_rows(dtype, d):
    """x, g and z as column blocks of one buffer; an odd width puts the blocks at
    odd offsets."""
    x, g, z, rate, bias = _inputs((2, 150, d), dtype, d, strided=True)
    assert not x.is_contiguous()
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias)
    _check_scan(Reference(x, g, z, rate, bias), out, hf, "strided")
    alone, h2 = jamba_ssm_gated_scan(x.contiguous(), g.contiguous(), z=z.contiguous(), rate=rate,
                                     bias=bias)
    assert_within(alone, out.double().cpu(), 0 * out.double().cpu() + 1e-2, "contiguous")
    one = jamba_ssm_gated_scan(x[:, :1], g[:, :1], z=z[:, :1], rate=rate, bias=bias)[0]
    assert torch.equal(one, out[:, :1])


@pytest.mark.parametrize("dtype,d,strides", [
    (F32, 1, (1, 1, 1)), (F32, 2, (5, 2, 7)), (F32, 3, (3, 6, 3)), (F32, 31, (31, 33, 34)),
    (F32, 33, (39, 33, 33)), (F32, 515, (515, 517, 518)), (F32, 130, (130, 130, 131)),
    (BF, 2, (2, 2, 2)), (BF, 6, (6, 10, 8)), (BF, 62, (62, 64, 66)), (BF, 1026, (1026, 1028, 1030)),
])
@pytest.mark.parametrize("batch,seqlen", [(1, 1), (1, 130), (70, 97)])
def test_rows_at_any_multiple_of_4_bytes(dtype, d, strides, batch, seqlen):
    """x, g and z with their own row strides, in buffers whose every other byte is a
    NaN: rows behind the last, channels past the width, and what lies between."""
    dev, rows = _dev(), batch * seqlen
    gen = torch.Generator(device=dev)
    gen.manual_seed(d)
    views = []
    for s in strides:
        buf = torch.full(((rows + 2) * s + d,), float("nan"), device=dev, dtype=dtype)
        v = buf.as_strided((batch, seqlen, d), (seqlen * s, s, 1))
        v.copy_(torch.randn(batch, seqlen, d, generator=gen, device=dev))
        views.append(v)
    x, g, z = views
    h0 = torch.randn(batch, d, generator=gen, device=dev)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, h0=h0)
    _check_scan(Reference(x, g, z, h0=h0), out, hf, f"{dtype} {d} {strides}")
    # the same rows as packed sequences of other lengths
    cu = sorted({0, rows // 3, rows // 2, rows})
    px, pg, pz = (v.as_strided((rows, d), (s, 1)) for v, s in zip(views, strides))
    out, hf = jamba_ssm_gated_scan(px, pg, z=pz,
                                   cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev))
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        ref = Reference(px[None, lo:hi], pg[None, lo:hi], pz[None, lo:hi])
        assert_within(out[lo:hi][None], ref.out, ref.e_out, f"sequence {i}")
        assert_within(hf[i:i + 1], ref.h_final, ref.e_final, f"state {i}")


LENGTHS = [0, 1, 63, 64, 65, 700, 0, 17, 128, 2]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [48, 75])
def test_packed_sequences_and_rows_behind_the_last(dtype, d):
    total = sum(LENGTHS)
    x, g, z, rate, bias = _inputs((total + 9, d), dtype, 5, strided=True, slow=True)
    dev = x.device
    cu = torch.tensor([0] + list(torch.tensor(LENGTHS).cumsum(0)), dtype=torch.int32, device=dev)
    h0 = torch.randn(len(LENGTHS), d, device=dev)
    out = torch.full((total + 9, d), 3.0, dtype=dtype, device=dev)
    jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0, cu_seqlens=cu, out=out)
    _, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0, cu_seqlens=cu)
    ref = Reference(x, g, z, rate, bias, h0, cu=cu.tolist())
    assert_within(out[:total], ref.out[:total], ref.e_out[:total], "packed out")
    assert_within(hf, ref.h_final, ref.e_final, "packed h_final")
    assert (out[total:] == 3.0).all(), "rows behind the last sequence were written"
    assert torch.equal(hf[0], h0[0]) and torch.equal(hf[6], h0[6])  # empty sequences


@pytest.mark.parametrize("n", [127, 128, 129, 300])
def test_more_packed_sequences_than_threads(n):
    """Up to 128 sequences are taken longest first, more in their order."""
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 40, (n,), generator=gen)
    lens[n // 2] = 333
    lens[0] = 0
    total, d = int(lens.sum()), 40
    x, g, z, rate, bias = _inputs((total, d), F32, n)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).int().to(x.device)
    h0, dh = torch.randn(n, d, device=x.device), torch.randn(n, d, device=x.device)
    dout = torch.randn(total, d, device=x.device)
    ref = Reference(x, g, z, rate, bias, h0, cu=cu.tolist())
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0, cu_seqlens=cu)
    _check_scan(ref, out, hf, f"{n} sequences")
    got = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias, h0=h0, dh_final=dh,
                                   cu_seqlens=cu)
    for k, (v, e) in ref.gradients(dout, dh).items():
        assert_within(got[k], v, e, k)


def test_offsets_past_the_rows_are_clamped():
    x, g, z, rate, bias = _inputs((50, 32), F32, 2)
    cu = torch.tensor([-5, 20, 70, 1000], dtype=torch.int32, device=x.device)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, cu_seqlens=cu)
    ref = Reference(x, g, z, rate, bias, cu=[0, 20, 50, 50])
    _check_scan(ref, out, hf, "clamped")
    back = torch.tensor([30, 10, 50], dtype=torch.int32, device=x.device)  # not increasing
    out, hf = jamba_ssm_gated_scan(x, g, cu_seqlens=back)
    assert (hf[0] == 0).all()  # an empty sequence


def test_state_slots():
    dev = _dev()
    lens, d, slots = [5, 0, 70, 1, 130], 66, 9
    x, g, z, rate, bias = _inputs((sum(lens), d), BF, 11)
    cu = torch.tensor([0, 5, 5, 75, 76, 206], dtype=torch.int32, device=dev)
    cache = torch.randn(slots, d, device=dev)
    before = cache.clone()
    # final rows; -1 and one past the cache are not written
    state = torch.tensor([3, 8, -1, 0, 9], dtype=torch.int32, device=dev)
    first = torch.tensor([-1, 8, 2, 0, 5], dtype=torch.int32, device=dev)
    ws = torch.zeros(16, dtype=torch.uint8, device=dev)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=cache, h_final=cache,
                                   cu_seqlens=cu, state_indices=state, initial_indices=first,
                                   workspace=ws)
    assert hf is cache
    assert jamba_ssm_gated_get_status(workspace=ws) == _lib.ERR_INVALID_ARG
    assert jamba_ssm_gated_get_status(workspace=ws) == 0  # cleared
    assert jamba_ssm_gated_get_status() == 0  # the library's own word is another
    h0 = torch.stack([torch.zeros(d, device=dev), before[8], before[2], before[0], before[5]])
    ref = Reference(x, g, z, rate, bias, h0, cu=cu.tolist())
    assert_within(out, ref.out, ref.e_out, "slots out")
    for b, row in ((0, 3), (1, 8), (3, 0)):
        assert_within(cache[row], ref.h_final[b], ref.e_final[b], f"cache row {row}")
    for row in (1, 2, 4, 5, 6, 7):
        assert torch.equal(cache[row], before[row])
    # without initial_indices the state row is read
    c2 = before.clone()
    s2 = torch.tensor([3, 8, 1, 0, 5], dtype=torch.int32, device=dev)
    out, _ = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=c2, h_final=c2,
                                  cu_seqlens=cu, state_indices=s2)
    ref = Reference(x, g, z, rate, bias, before[s2.long()], cu=cu.tolist())
    assert_within(out, ref.out, ref.e_out, "slots out, own rows")
    assert_within(c2[s2.long()], ref.h_final, ref.e_final, "slots state, own rows")
    assert jamba_ssm_gated_get_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_at_the_ends_of_their_range(dtype):
    """Gates that open fully, close fully and to the last bit: u = rate, u = 0."""
    x, g, z, rate, bias = _inputs((1, 90, 64), dtype, 1)
    g[0, ::3] = 60.0
    g[0, 1::5] = -60.0
    g[0, 2::7, ::2] = float("inf")
    g[0, 3::7, ::2] = float("-inf")
    z[0, ::4] = 90.0
    z[0, 1::4] = -90.0
    rate[:8], rate[8:16] = 0.0, 1.0
    h0 = torch.randn(1, 64, device=x.device)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, h0=h0)
    gf = g.float().clamp(-1e4, 1e4)  # the bound's |v|; sigmoid is 0 or 1 there
    ref = Reference(x, gf.to(F32), z, rate, None, h0)
    ref.e_out = ref.e_out + (2.0 ** -8 if dtype == BF else 0) * ref.out.abs()
    _check_scan(ref, out, hf, "saturated")


def test_slow_channels_keep_their_memory():
    """rate 1e-6 over 5000 tokens: the state moves by the sum of tiny updates,
    which a decay rounded to 1 - 1e-6 would miss by 3%."""
    dev = _dev()
    x = torch.ones(1, 5000, 8, device=dev)
    g = torch.zeros(1, 5000, 8, device=dev)
    rate = torch.full((8,), 1e-6, device=dev)
    _, hf = jamba_ssm_gated_scan(x, g, rate=rate)
    r = float(torch.tensor(1e-6)) * 0.5
    want = 1 - (1 - r) ** 5000
    # each step rounds h (at most 2.5e-3, so by 2^-33) once or twice, and u by 2^-21
    assert abs(float(hf[0, 0].double()) - want) < 5000 * 2.0 ** -32 + want * 2.0 ** -20


def test_non_finite_input_stays_in_its_channel_and_its_future():
    x, g, z, rate, bias = _inputs((2, 300, 64), F32, 4)
    clean, _ = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias)
    y = x.clone()
    y[0, 130, 5] = float("nan")
    y[1, 0, 9] = float("inf")
    out, hf = jamba_ssm_gated_scan(y, g, z=z, rate=rate, bias=bias)
    mask = torch.zeros_like(out, dtype=torch.bool)
    mask[0, 130:, 5] = True
    mask[1, :, 9] = True
    assert torch.equal(out[~mask], clean[~mask])
    assert not torch.isfinite(out[0, 130:, 5]).any() and not torch.isfinite(hf[0, 5])
    # rows behind a packed sequence may hold anything
    rows = torch.full((140, 64), float("nan"), device=x.device)
    rows[:100] = x[0, :100]
    gr = rows.clone()
    gr[:100] = g[0, :100]
    cu = torch.tensor([0, 33, 100], dtype=torch.int32, device=x.device)
    out, hf = jamba_ssm_gated_scan(rows, gr, rate=rate, cu_seqlens=cu)
    assert torch.isfinite(out[:100]).all() and torch.isfinite(hf).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,seqlen,d,gate", [
    (1, 1, 1, True), (2, 1, 64, False), (1, 9, 5, True), (2, 64, 64, True), (3, 65, 33, False),
    (1, 127, 128, True), (2, 300, 70, True), (1, 1100, 34, True), (2, 513, 24, False),
])
def test_backward_matches_formulas(dtype, batch, seqlen, d, gate):
    x, g, z, rate, bias = _inputs((batch, seqlen, d), dtype, 3 * d + seqlen, gate=gate)
    dev = x.device
    h0, dh = torch.randn(batch, d, device=dev), torch.randn(batch, d, device=dev)
    dout = torch.randn(batch, seqlen, d, device=dev).to(dtype)
    ref = Reference(x, g, z, rate, bias, h0)
    want = ref.gradients(dout, dh)
    ckpt = jamba_ssm_gated_scan_ckpt(x)
    assert ckpt.numel() * 4 == jamba_ssm_gated_scan_ckpt_size(batch, batch * seqlen, d)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0, ckpt=ckpt)
    _check_scan(ref, out, hf, "with checkpoints")
    plain, _ = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0)
    assert torch.equal(plain, out)
    with_ck = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias, h0=h0, dh_final=dh,
                                       ckpt=ckpt)
    without = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias, h0=h0, dh_final=dh)
    for k, (v, e) in want.items():
        if v is None:
            assert with_ck[k] is None
            continue
        assert_within(with_ck[k], v, e, k)
        assert torch.equal(with_ck[k], without[k]), f"{k} depends on who made the checkpoints"


@pytest.mark.parametrize("dtype,batch,seqlen,d", [(BF, 24, 300, 320), (BF, 40, 100, 520),
                                                  (F32, 24, 150, 310)])
def test_backward_of_many_tiles(dtype, batch, seqlen, d):
    """The cuts without clusters, from the forward's checkpoints."""
    x, g, z, rate, bias = _inputs((batch, seqlen, d), dtype, d)
    dev = x.device
    h0, dh = torch.randn(batch, d, device=dev), torch.randn(batch, d, device=dev)
    dout = torch.randn(batch, seqlen, d, device=dev).to(dtype)
    ckpt = jamba_ssm_gated_scan_ckpt(x)
    jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0, ckpt=ckpt)
    got = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias, h0=h0, dh_final=dh,
                                   ckpt=ckpt)
    for k, (v, e) in Reference(x, g, z, rate, bias, h0).gradients(dout, dh).items():
        assert_within(got[k], v, e, k)


@pytest.mark.parametrize("dtype,d", [(BF, 50), (F32, 33), (BF, 64)])
def test_backward_of_packed_strided_sequences(dtype, d):
    total = sum(LENGTHS)
    x, g, z, rate, bias = _inputs((total + 4, d), dtype, 6, strided=True)
    dev = x.device
    n = len(LENGTHS)
    cu = torch.tensor([0] + list(torch.tensor(LENGTHS).cumsum(0)), dtype=torch.int32, device=dev)
    h0, dh = torch.randn(n, d, device=dev), torch.randn(n, d, device=dev)
    dout = torch.randn(total + 4, d, device=dev).to(dtype)
    ckpt = jamba_ssm_gated_scan_ckpt(x, cu_seqlens=cu)
    jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, h0=h0, cu_seqlens=cu, ckpt=ckpt)
    got = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias, h0=h0, dh_final=dh,
                                   cu_seqlens=cu, ckpt=ckpt)
    want = Reference(x, g, z, rate, bias, h0, cu=cu.tolist()).gradients(dout, dh)
    for k, (v, e) in want.items():
        if k in ("dx", "dg", "dz"):
            assert_within(got[k][:total], v[:total], e[:total], k)
        else:
            assert_within(got[k], v, e, k)
    assert torch.equal(got["dh0"][0], dh[0])  # an empty sequence hands its gradient on
    bare = jamba_ssm_gated_scan_bwd(x, g, dout, cu_seqlens=cu)
    assert bare["dz"] is None and bare["drate"] is None and bare["dbias"] is None
    want = Reference(x, g, cu=cu.tolist()).gradients(dout)
    for k in ("dx", "dg"):
        assert_within(bare[k][:total], want[k][0][:total], want[k][1][:total], "bare " + k)


def test_backward_of_nothing():
    dev = _dev()
    e = lambda *s: torch.empty(*s, device=dev)  # noqa: E731
    rate = torch.ones(8, device=dev)
    out, hf = jamba_ssm_gated_scan(e(2, 0, 8), e(2, 0, 8), rate=rate, h0=torch.ones(2, 8, device=dev))
    assert out.shape == (2, 0, 8) and (hf == 1).all()
    got = jamba_ssm_gated_scan_bwd(e(2, 0, 8), e(2, 0, 8), e(2, 0, 8), rate=rate,
                                   dh_final=torch.full((2, 8), 2.0, device=dev))
    assert (got["dh0"] == 2).all() and (got["drate"] == 0).all()
    got = jamba_ssm_gated_scan_bwd(e(0, 5, 8), e(0, 5, 8), e(0, 5, 8), rate=rate)
    assert (got["drate"] == 0).all() and got["dh0"].shape == (0, 8)


def test_neighbours_and_what_memory_held_change_no_bits():
    """A channel pair's results are its own inputs' alone: not those of the other
    lanes of its warp, which may have to do their rows again, nor what shared
    memory held for lanes past the width."""
    x, g, z, rate, bias = _inputs((1, 1100, 34), BF, 8)
    dout = torch.randn(x.shape, device=x.device).to(BF)
    one, _ = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias)
    back = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias)
    dirty = torch.full((64, 512, 512), float("nan"), dtype=BF, device=x.device)
    g2 = g.clone()
    g2[0, ::7, 6:8] = -80.0  # one pair whose exponentials' product overflows
    g2[0, 5, 20] = float("nan")
    keep = [c for c in range(34) if c not in (6, 7, 20, 21)]
    for _ in range(4):
        jamba_ssm_gated_scan(dirty, dirty)  # leaves NaN behind
        out, _ = jamba_ssm_gated_scan(x, g2, z=z, rate=rate, bias=bias)
        assert torch.equal(out[..., keep], one[..., keep])
        got = jamba_ssm_gated_scan_bwd(x, g2, dout, z=z, rate=rate, bias=bias)
        for k, v in got.items():
            assert torch.equal(v[..., keep], back[k][..., keep]), k


def test_gradients_of_runs_are_the_same_bits():
    x, g, z, rate, bias = _inputs((3, 700, 160), BF, 12)
    dout = torch.randn(x.shape, device=x.device).to(BF)
    one = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias)
    for _ in range(3):
        two = jamba_ssm_gated_scan_bwd(x, g, dout, z=z, rate=rate, bias=bias)
        for k in one:
            assert one[k] is None or torch.equal(one[k], two[k]), k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,d,gate", [(1, 1, True), (3, 33, False), (5, 64, True),
                                          (17, 1000, True), (2, 4096, False)])
def test_update_matches_recurrence(dtype, batch, d, gate):
    x, g, z, rate, bias = _inputs((batch, d), dtype, d, gate=gate, strided=batch > 4)
    state = torch.randn(batch, d, device=x.device)
    ref = Reference(x[:, None], g[:, None], None if z is None else z[:, None], rate, bias, state)
    out = jamba_ssm_gated_state_update(state, x, g, z=z, rate=rate, bias=bias)
    assert_within(out, ref.out, ref.e_out, "update out")
    assert_within(state, ref.h_final, ref.e_final, "update state")


def test_update_slots_and_padding():
    dev = _dev()
    x, g, z, rate, bias = _inputs((6, 72), BF, 8)
    cache = torch.randn(10, 72, device=dev)
    before = cache.clone()
    idx = torch.tensor([9, -1, 4, 10, 0, -7], dtype=torch.int32, device=dev)
    out = torch.full((6, 72), 5.0, dtype=BF, device=dev)
    ws = torch.zeros(16, dtype=torch.uint8, device=dev)
    jamba_ssm_gated_state_update(cache, x, g, z=z, rate=rate, bias=bias, out=out,
                                 state_indices=idx, workspace=ws)
    assert jamba_ssm_gated_get_status(workspace=ws) == _lib.ERR_INVALID_ARG
    keep = [0, 2, 4]
    rows = idx[keep].long()
    ref = Reference(x[keep][:, None], g[keep][:, None], z[keep][:, None], rate, bias, before[rows])
    assert_within(out[keep], ref.out, ref.e_out, "slots out")
    assert_within(cache[rows], ref.h_final, ref.e_final, "slots state")
    assert (out[[1, 3, 5]] == 5).all()
    rest = [r for r in range(10) if r not in rows.tolist()]
    assert torch.equal(cache[rest], before[rest])


def test_updates_continue_a_scan():
    x, g, z, rate, bias = _inputs((2, 40, 64), F32, 9)
    want, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias)
    # batched sequences follow one another without a gap: a part of each is copied
    part = [t[:, :25].contiguous() for t in (x, g, z)]
    _, state = jamba_ssm_gated_scan(part[0], part[1], z=part[2], rate=rate, bias=bias)
    ref = Reference(x, g, z, rate, bias)
    for t in range(25, 40):
        out = jamba_ssm_gated_state_update(state, x[:, t], g[:, t], z=z[:, t], rate=rate, bias=bias)
        rows = [t, 40 + t]
        assert_within(out, ref.out[rows], ref.e_out[rows], f"step {t}")
    assert_within(state, ref.h_final, ref.e_final, "last state")


def test_offsets_past_32_bits():
    """2.2e9 elements in each activation and 2.2e9 in the state cache: the far end
    is that of the same rows taken alone."""
    dev, rows, d, cut = _dev(), 270_000, 8192, 269_000
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    x = torch.randn(1, rows, d, generator=gen, device=dev, dtype=BF)
    g = torch.randn(1, rows, d, generator=gen, device=dev, dtype=BF)
    out, hf = jamba_ssm_gated_scan(x, g)
    _, h = jamba_ssm_gated_scan(x[:, :cut], g[:, :cut])
    tail, ht = jamba_ssm_gated_scan(x[:, cut:], g[:, cut:], h0=h)
    # both are within the recurrence's bound, 2^-21 of the largest |x| for each of the
    # about 10 steps that a gate near 1/2 remembers, and half a bf16 step
    assert ((tail - out[:, cut:]).abs().float() <= 2.0 ** -7 * tail.abs().float() + 1e-3).all()
    assert (ht - hf).abs().max() < 1e-3
    dout = torch.ones_like(x)
    grads = jamba_ssm_gated_scan_bwd(x, g, dout)
    part = jamba_ssm_gated_scan_bwd(x[:, cut:], g[:, cut:], dout[:, cut:], h0=h)
    for k in ("dx", "dg"):
        a, b = grads[k][:, cut:].float(), part[k].float()
        assert ((a - b).abs() <= 2.0 ** -6 * b.abs() + 1e-3).all(), k
    del out, tail, grads, part, dout
    big = torch.zeros(270_000, 8192, device=dev)
    idx = torch.tensor([269_999, 3], dtype=torch.int32, device=dev)
    y = jamba_ssm_gated_state_update(big, x[0, :2], g[0, :2], state_indices=idx)
    small = torch.zeros(2, 8192, device=dev)
    want = jamba_ssm_gated_state_update(small, x[0, :2], g[0, :2])
    assert torch.equal(y, want) and torch.equal(big[idx.long()], small)
    assert int(torch.count_nonzero(big[4:269_999])) == 0


def test_graph_streams_and_two_calls_at_once():
    """Captured and replayed on new inputs, beside an eager call on another
    stream: the two share nothing."""
    dev = _dev()
    x, g, z, rate, bias = _inputs((2, 400, 136), BF, 21)
    dout = torch.randn(x.shape, device=dev).to(BF)
    static = [t.clone() for t in (x, g, z, dout)]

    def step(a, b, c, d):
        ck = jamba_ssm_gated_scan_ckpt(a)
        out, hf = jamba_ssm_gated_scan(a, b, z=c, rate=rate, bias=bias, ckpt=ck)
        return {"out": out, "hf": hf, **jamba_ssm_gated_scan_bwd(a, b, d, z=c, rate=rate,
                                                                bias=bias, ckpt=ck)}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(*static)
    y, h, w, e = (t.flip(1).contiguous() for t in (x, g, z, dout))
    for s, t in zip(static, (y, h, w, e)):
        s.copy_(t)
    torch.cuda.synchronize()
    want_new, want_old = step(y, h, w, e), step(x, g, z, dout)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        eager = step(x, g, z, dout)
    graph.replay()
    torch.cuda.synchronize()
    for k in kept:
        assert torch.equal(kept[k], want_new[k]), k
        assert torch.equal(eager[k], want_old[k]), k
    # a stream named by the caller
    out, _ = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, stream=side)
    side.synchronize()
    assert torch.equal(out, want_old["out"])
    out, _ = jamba_ssm_gated_scan(x, g, z=z, rate=rate, bias=bias, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want_old["out"])


def test_refusals():
    x, g, z, rate, bias = _inputs((2, 10, 16), F32, 1)
    for call in (lambda: jamba_ssm_gated_scan(x, None),
                 lambda: jamba_ssm_gated_scan_bwd(x, g, None),
                 lambda: jamba_ssm_gated_state_update(None, x[0], g[0])):
        with pytest.raises(TypeError, match="torch.Tensor"):
            call()
    with pytest.raises(ValueError, match="CUDA"):
        jamba_ssm_gated_scan(x.cpu(), g.cpu())
    with pytest.raises(TypeError):
        jamba_ssm_gated_scan(x.half(), g.half())
    with pytest.raises(TypeError):
        jamba_ssm_gated_scan(x, g.to(BF))
    with pytest.raises(ValueError, match="shape"):
        jamba_ssm_gated_scan(x, g[:, :5])
    with pytest.raises(ValueError, match="rows"):
        jamba_ssm_gated_scan(x, g.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="rows"):
        jamba_ssm_gated_scan(x, g[:, :1].expand(2, 10, 16))
    with pytest.raises(ValueError, match="rows"):  # a gap between the sequences
        jamba_ssm_gated_scan(x[:, :5], g[:, :5])
    with pytest.raises(ValueError, match="rows"):
        jamba_ssm_gated_scan(x, torch.randn(2, 10, 32, device=x.device)[..., ::2])
    with pytest.raises(ValueError, match="shape"):
        jamba_ssm_gated_scan(x, g, rate=rate[:8])
    with pytest.raises(TypeError):
        jamba_ssm_gated_scan(x, g, rate=rate.double())
    idx = torch.zeros(2, dtype=torch.int32, device=x.device)
    with pytest.raises(ValueError, match="initial_indices"):
        jamba_ssm_gated_scan(x, g, initial_indices=idx)
    with pytest.raises(ValueError, match="cache"):
        jamba_ssm_gated_scan(x, g, state_indices=idx)
    with pytest.raises(_lib.JambaSSMError):
        jamba_ssm_gated_scan(x, g, out=x)
    with pytest.raises(_lib.JambaSSMError):
        jamba_ssm_gated_state_update(torch.zeros(10, 16, device=x.device), x[0], g[0], out=g[0])
    ws = torch.empty(8, dtype=torch.uint8, device=x.device)
    with pytest.raises(_lib.JambaSSMError):
        jamba_ssm_gated_scan_bwd(x, g, x.clone(), workspace=ws)


_SLOW = (2.0 ** -24, 1e-6, 1e-5, 1e-4)  # u is half of it: from below a half step of 1 on


@pytest.mark.parametrize("dtype,batch,seqlen,d", [
    (F32, 1, 16384, 8), (BF, 1, 16384, 64), (BF, 2, 8192, 33), (F32, 230, 8192, 32),
    (F32, 300, 4096, 32), (BF, 1, 16000, 1024)])
def test_slow_channels_stay_at_their_input(dtype, batch, seqlen, d):
    """A state equal to its input does not move, however little a row forgets.

    A run's decay n = P - 1 and its b have relative errors of 2 roundings a row and 2 a
    join: at most (32 + 2 * 19) 2^-24 each, so n c + b, which is 0, is within 2^-16 c of
    the run's own decay, and a state within 2^-16 c of its input stays there: rounding
    to nearest keeps a value that moves towards c on its side of it.  A decay that is
    rounded row by row moves the state by up to 2^-25 c a row instead."""
    dev = _dev()
    c = torch.linspace(0.6, 1.9, d, device=dev).to(dtype)
    x = c.expand(batch, seqlen, d).contiguous()
    g = torch.zeros_like(x)
    rate = torch.tensor(_SLOW, device=dev).repeat(-(-d // 4))[:d].contiguous()
    h0 = c.float().expand(batch, d).contiguous()
    z = torch.ones_like(x) if dtype == F32 else None
    ckpt = jamba_ssm_gated_scan_ckpt(x)
    out, hf = jamba_ssm_gated_scan(x, g, z=z, rate=rate, h0=h0, ckpt=ckpt)
    off = ((hf - h0).abs() / h0).amax(0)
    assert (off <= 2.0 ** -16).all(), off[:4]
    at = ckpt.reshape(-1, d)[: seqlen // 64]
    assert ((at - h0[0]).abs() <= 2.0 ** -16 * h0[0]).all()
    # a row's own state has the row-by-row error of its run, 16 roundings of P and of b
    gate = 1.0 if z is None else torch.sigmoid(torch.ones((), dtype=torch.float64, device=dev))
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -22  # fp32: three roundings of the gate
    assert ((out.double() / gate - h0.double()[:, None]).abs()
            <= (2.0 ** -16 + 2.0 ** -19 + half) * h0[:, None]).all()


@pytest.mark.parametrize("dtype,batch,seqlen,d", [
    (F32, 1, 16384, 8), (BF, 1, 16384, 64), (BF, 2, 8192, 33), (F32, 300, 8192, 32)])
def test_slow_channels_forget_at_their_rate(dtype, batch, seqlen, d):
    """Forwards without input, and the gradient of h0 without dout: (1 - u)^rows.

    A run rounds the state once, by 2^-24 of it at most, and its decay, 70 roundings of
    itself (above): rows / 8 2^-24 and 2^-17 (1 - (1 - u)^rows) in all."""
    dev = _dev()
    x = torch.zeros(batch, seqlen, d, dtype=dtype, device=dev)
    rate = torch.tensor(_SLOW, device=dev).repeat(-(-d // 4))[:d].contiguous()
    one = torch.ones(batch, d, device=dev)
    ckpt = jamba_ssm_gated_scan_ckpt(x)
    _, hf = jamba_ssm_gated_scan(x, x, rate=rate, h0=one, ckpt=ckpt)
    grads = jamba_ssm_gated_scan_bwd(x, x, x, rate=rate, h0=one, dh_final=one, ckpt=ckpt)
    want = (1 - rate.double() / 2) ** seqlen
    bound = seqlen / 8 * 2.0 ** -24 + 2.0 ** -17
    for got, what in ((hf, "h_final"), (grads["dh0"], "dh0")):
        off = (got.double() - want).abs().amax(0)
        assert (off <= bound).all(), (what, off[:4], bound)


@pytest.mark.parametrize("seqlen", [1, 16, 63, 100, 120])
def test_fast_channels_forget_exactly(seqlen):
    """u = 1/2: every product is a power of two, and nothing of a state is left but that."""
    dev = _dev()
    x = torch.zeros(2, seqlen, 40, device=dev)
    h0 = torch.linspace(1, 3e4, 40, device=dev).repeat(2, 1)
    ckpt = jamba_ssm_gated_scan_ckpt(x)
    out, hf = jamba_ssm_gated_scan(x, x, h0=h0, ckpt=ckpt)
    grads = jamba_ssm_gated_scan_bwd(x, x, x, h0=h0, dh_final=h0, ckpt=ckpt)
    want = h0 * 2.0 ** -seqlen
    assert torch.equal(hf, want) and torch.equal(out[:, -1], want)
    assert torch.equal(grads["dh0"], want)
