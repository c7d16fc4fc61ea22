"""The maps of a continuous batch on the GPU against a plain loop over requests,
and a whole serving run: maps, 8-bit projections, packed scans and decode steps."""
import random

import pytest
import torch

from selective_state_space_26_b200 import (_lib, jamba_ssm_batch_maps, jamba_ssm_gated_scan,
                                           jamba_ssm_gated_state_update, jamba_ssm_i8_proj,
                                           jamba_ssm_i8_quant, jamba_ssm_serve_get_status)
from tests.gated_ref import Reference, assert_within

pytestmark = pytest.mark.gpu


def _i32(v):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def maps_ref(new, ctx, table, free, slots, free_slots, bs, rows):
    """The header's definition, request by request; (maps, whether something did not fit)."""
    width = len(table[0]) if table else 1
    table, slots = [list(r) for r in table], list(slots)
    pos, req, smap = [-1] * rows, [-1] * rows, [-1] * rows
    cu, state, first = [0], [], []
    blocks = taken = longest = 0
    bad = False
    for b, want in enumerate(new):
        want, c = max(want, 0), max(ctx[b], 0)
        n = min(want, rows - cu[-1])
        had = min(-(-c // bs), width)
        need = -(-(c + n) // bs) if n else had
        bad |= n < want or need > width
        for j in range(had, min(need, width)):
            ok = blocks < len(free)
            table[b][j] = free[blocks] if ok else -1
            bad |= not ok
            blocks += 1
        if n and c == 0:
            ok = taken < len(free_slots)
            slots[b] = free_slots[taken] if ok else -1
            bad |= not ok
            taken += 1
        state.append(slots[b] if n else -1)
        first.append(slots[b] if n and c else -1)
        for i in range(n):
            t, p = cu[-1] + i, c + i
            blk = table[b][p // bs] if p // bs < width else -1
            pos[t], req[t] = p, b
            smap[t] = blk * bs + p % bs if blk >= 0 else -1
        longest = max(longest, n)
        cu.append(cu[-1] + n)
    return {"cu_seqlens": cu, "positions": pos, "token_request": req, "slot_map": smap,
            "block_tables": table, "request_slots": slots, "state_indices": state,
            "initial_indices": first,
            "counts": [cu[-1], min(blocks, len(free)), min(taken, len(free_slots)), longest]}, bad


def _run(new, ctx, table, free, slots, free_slots, bs, rows):
    got = jamba_ssm_batch_maps(_i32(new), _i32(table).view(len(new), -1), _i32(free), _i32(slots),
                               _i32(free_slots), ctx_lens=None if ctx is None else _i32(ctx),
                               block_size=bs, max_tokens=rows)
    return {k: v.tolist() for k, v in got.items()}


def _case(rng, requests, most, bs, ctx_most=100, spare=5, rows=None):
    new = [rng.choice((0, 1, 1, rng.randint(1, most))) for _ in range(requests)]
    ctx = [rng.choice((0, rng.randint(1, ctx_most))) for _ in range(requests)]
    width = max([1] + [-(-(c + n) // bs) for c, n in zip(ctx, new)])
    ids = list(range(requests * width + spare))
    rng.shuffle(ids)
    table = [[-1] * width for _ in range(requests)]
    for b in range(requests):
        for j in range(-(-ctx[b] // bs)):
            table[b][j] = ids.pop()
    slot_ids = list(range(2 * requests + 1))
    rng.shuffle(slot_ids)
    slots = [slot_ids.pop() if c else -1 for c in ctx]
    return new, ctx, table, ids, slots, slot_ids, bs, sum(new) + 7 if rows is None else rows


@pytest.mark.parametrize("requests,most,bs", [(1, 1, 16), (1, 300, 16), (3, 40, 1), (31, 20, 7),
                                              (64, 5, 64), (257, 9, 16), (1000, 30, 32),
                                              (2500, 3, 16), (70, 1500, 100)])
def test_maps_match_the_loop(requests, most, bs):
    args = _case(random.Random(requests + most), requests, most, bs)
    want, bad = maps_ref(*args)
    assert not bad
    assert _run(*args) == want
    assert jamba_ssm_serve_get_status() == 0


def test_no_requests_no_tokens_and_no_context():
    got = jamba_ssm_batch_maps(_i32([]), _i32([]).view(0, 4), _i32([1]), _i32([]), _i32([]),
                               max_tokens=5)
    assert got["cu_seqlens"].tolist() == [0] and got["counts"].tolist() == [0, 0, 0, 0]
    assert got["slot_map"].tolist() == [-1] * 5 and got["positions"].tolist() == [-1] * 5
    args = ([0, 0], [5, 0], [[7, 9], [3, 3]], [1], [4, -1], [2], 4, 0)
    want, _ = maps_ref(*args)
    assert _run(*args) == want
    new = [3, 0, 2]
    want, _ = maps_ref(new, [0] * 3, [[9, 9]] * 3, [1, 2, 3], [-1] * 3, [5, 6], 2, 6)
    assert _run(new, None, [[9, 9]] * 3, [1, 2, 3], [-1] * 3, [5, 6], 2, 6) == want
    assert jamba_ssm_serve_get_status() == 0


@pytest.mark.parametrize("case", [
    # tokens past max_tokens: the request in the middle is cut, the ones behind get none
    ([5, 6, 7, 1], [0, 3, 0, 9], [[0, 0, 0, 0]] * 4, list(range(20, 40)), [-1, 3, -1, 4], [8, 9], 4, 9),
    # too few free blocks
    ([9, 9], [0, 0], [[-1] * 3] * 2, [11, 12, 13, 14], [-1, -1], [1, 2], 4, 18),
    # no free block at all, none of the list
    ([2], [0], [[-1]], [], [-1], [], 4, 2),
    # too few state slots
    ([1, 1, 1], [0, 0, 0], [[-1]] * 3, [1, 2, 3], [-1] * 3, [7], 4, 3),
    # a request longer than its table; one whose context already is
    ([9, 2], [0, 20], [[-1, -1], [5, 6]], [1, 2, 3, 4, 5], [-1, 3], [7], 4, 11),
    # negative lengths count as none; a negative block in the table
    ([-4, 3, 2], [2, -9, 5], [[1, 1], [-1, -1], [3, -1]], [4, 5, 6], [0, -1, 2], [9], 4, 8),
])
def test_what_does_not_fit_is_recorded(case):
    want, bad = maps_ref(*case)
    assert _run(*case) == want
    assert jamba_ssm_serve_get_status() == (_lib.ERR_INVALID_ARG if bad else 0)
    assert jamba_ssm_serve_get_status() == 0


def test_many_requests_and_long_maps():
    rng = random.Random(4)
    args = _case(rng, 20000, 6, 8, ctx_most=30)
    want, bad = maps_ref(*args)
    assert not bad and _run(*args) == want
    new, ctx = [200000, 1, 70000], [0, 500000, 3]
    bs = 1000
    table = [[-1] * 501 for _ in new]
    for j in range(500):
        table[1][j] = 5000 + j
    table[2][0] = 4999
    args = (new, ctx, table, list(range(400)), [-1, 0, 1], [5], bs, 270100)
    want, bad = maps_ref(*args)
    assert not bad and _run(*args) == want


@pytest.mark.parametrize("requests", [2, 2100])  # either form of the call
@pytest.mark.parametrize("bs,width", [(16, 4), (1 << 20, 1 << 11), (1, 3)])
def test_positions_past_31_bits(requests, bs, width):
    """A context of 2^31 - 3 tokens has three positions left: the tokens behind
    have none, touch no table and are recorded; the request behind is whole."""
    ctx = _i32([2 ** 31 - 3, 0] + [5] * (requests - 2))
    new = _i32([6, 2] + [0] * (requests - 2))
    table = torch.full((requests, width), -7, dtype=torch.int32, device=ctx.device)
    table[0] = torch.arange(width, device=ctx.device) + 100
    maps = jamba_ssm_batch_maps(new, table, _i32([9, 8, 7]), _i32([-1] * requests), _i32([4]),
                                ctx_lens=ctx, block_size=bs, max_tokens=16)
    last = 2 ** 31 - 1
    assert maps["positions"].tolist() == [last - 2, last - 1, last, -1, -1, -1, 0, 1] + [-1] * 8
    assert maps["token_request"].tolist() == [0] * 6 + [1, 1] + [-1] * 8
    there = [(100 + (last - i) // bs) * bs + (last - i) % bs if (last - i) // bs < width else -1
             for i in (2, 1, 0)]
    second = [9, 8] if bs == 1 else [9 * bs, 9 * bs + 1]
    assert maps["slot_map"].tolist() == there + [-1] * 3 + second + [-1] * 8
    assert table[0].tolist() == list(range(100, 100 + width))
    taken = 2 if bs == 1 else 1
    assert table[1, :3].tolist() == ([9, 8] if bs == 1 else [9]) + [-7] * (3 - taken)
    assert maps["counts"].tolist() == [8, taken, 1, 6]
    assert jamba_ssm_serve_get_status() == _lib.ERR_INVALID_ARG


def test_tables_and_maps_past_32_bits():
    """2.7e9 table entries and 2^30 rows of the per-token maps."""
    requests, width, bs, rows = 160, 1 << 24, 16, 1 << 30
    table = torch.full((requests, width), -3, dtype=torch.int32, device=_i32([0]).device)
    new = [0] * requests
    new[1], new[-1] = rows - 40, 40
    blocks = -(-new[1] // bs) + 3
    free = torch.arange(blocks, dtype=torch.int32, device="cuda") + 5
    maps = jamba_ssm_batch_maps(_i32(new), table, free, _i32([-1] * requests), _i32([1, 0]),
                                block_size=bs, max_tokens=rows)
    # request 1 needs 2^26 blocks and has room for 2^24: recorded, the rest of it has no block
    assert jamba_ssm_serve_get_status() == _lib.ERR_INVALID_ARG
    assert maps["counts"].tolist() == [rows, width + 3, 2, rows - 40]
    assert maps["positions"][-41:].tolist() == [rows - 41] + list(range(40))
    assert maps["token_request"][-41:].tolist() == [1] + [requests - 1] * 40
    mine = free[width:width + 3]
    own = (mine.long()[:, None] * bs + torch.arange(bs, device="cuda")).flatten()[:40]
    assert torch.equal(maps["slot_map"][-40:], own)
    end = width * bs
    assert maps["slot_map"][end - 2:end + 2].tolist() == [(width + 4) * bs + 14, (width + 4) * bs + 15, -1, -1]
    assert torch.equal(table[-1, :4], torch.cat([mine, _i32([-3])]))
    assert torch.equal(table[1], free[:width])
    assert int((table[0] != -3).sum()) == 0 and int((table[2:-1] != -3).sum()) == 0


def test_graph_replays_on_new_lengths():
    rng = random.Random(6)
    new, ctx, table, free, slots, free_slots, bs, _ = _case(rng, 40, 30, 16)
    rows = 1300
    t = {k: _i32(v) for k, v in dict(new=new, ctx=ctx, table=table, free=free, slots=slots,
                                     fs=free_slots).items()}
    call = lambda: jamba_ssm_batch_maps(t["new"], t["table"], t["free"], t["slots"], t["fs"],  # noqa: E731
                                        ctx_lens=t["ctx"], block_size=bs, max_tokens=rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    fewer = [min(v, 3) for v in new]
    t["new"].copy_(_i32(fewer))
    t["table"].copy_(_i32(table))
    t["slots"].copy_(_i32(slots))
    graph.replay()
    torch.cuda.synchronize()
    want, bad = maps_ref(fewer, ctx, table, free, slots, free_slots, bs, rows)
    assert not bad and {k: v.tolist() for k, v in got.items()} == want


def test_refusals():
    n = _i32([1, 2])
    ok = dict(block_tables=_i32([[0], [1]]), free_blocks=n, request_slots=n.clone(), free_slots=n)
    with pytest.raises(ValueError, match="max_tokens"):
        jamba_ssm_batch_maps(n, **ok)
    with pytest.raises(ValueError, match="block_size"):
        jamba_ssm_batch_maps(n, **ok, max_tokens=3, block_size=0)
    with pytest.raises(TypeError):
        jamba_ssm_batch_maps(n.long(), **ok, max_tokens=3)
    with pytest.raises(ValueError, match="shape"):
        jamba_ssm_batch_maps(n, **{**ok, "request_slots": _i32([1])}, max_tokens=3)
    with pytest.raises(ValueError, match="CUDA"):
        jamba_ssm_batch_maps(n.cpu(), **ok, max_tokens=3)
    with pytest.raises(_lib.JambaSSMError):  # the slots read are the slots written
        jamba_ssm_batch_maps(n, **{**ok, "request_slots": ok["free_slots"]}, max_tokens=3)


def test_serving_run():
    """Three steps of a continuous batch through a recurrent layer in 8 bits: the
    maps, the input projection to x | g | z, the packed scan with state slots, the
    output projection; then a decode step through the one-token update.  Each
    request's outputs are those of its tokens alone, from zero."""
    rng = random.Random(2)
    gen = torch.Generator(device="cuda")
    _i32([0])
    gen.manual_seed(3)
    d_model, d, requests, bs, width = 96, 64, 5, 8, 16
    w_in, s_in = jamba_ssm_i8_quant(torch.randn(3 * d, d_model, generator=gen, device="cuda"))
    w_out, s_out = jamba_ssm_i8_quant(torch.randn(d_model, d, generator=gen, device="cuda"))
    rate = torch.rand(d, generator=gen, device="cuda")
    tokens = [torch.randn(60, d_model, generator=gen, device="cuda").to(torch.bfloat16)
              for _ in range(requests)]
    cache = torch.full((11, d), 77.0, device="cuda")  # what earlier requests left
    table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    slots = torch.full((requests,), -1, dtype=torch.int32, device="cuda")
    free_b, free_s = rng.sample(range(80), 80), rng.sample(range(11), 11)
    done = [0] * requests
    outs = [[] for _ in range(requests)]
    project = lambda v, w, s: jamba_ssm_i8_proj(*jamba_ssm_i8_quant(v), w, s)  # noqa: E731

    def mixer_inputs(flat):
        proj = project(flat, w_in, s_in)
        return proj[:, :d], proj[:, d:2 * d], proj[:, 2 * d:]

    for step in ([20, 0, 9, 1, 33], [5, 17, 0, 1, 2], [1, 1, 30, 1, 0]):
        flat = torch.cat([tokens[b][done[b]:done[b] + n] for b, n in enumerate(step)])
        maps = jamba_ssm_batch_maps(_i32(step), table, _i32(free_b), slots, _i32(free_s),
                                    ctx_lens=_i32(done), block_size=bs, max_tokens=flat.shape[0])
        x, g, z = mixer_inputs(flat)
        y, _ = jamba_ssm_gated_scan(x, g, z=z, rate=rate, h0=cache, h_final=cache,
                                    cu_seqlens=maps["cu_seqlens"],
                                    state_indices=maps["state_indices"],
                                    initial_indices=maps["initial_indices"])
        out = project(y, w_out, s_out)
        used = maps["counts"].tolist()
        free_b, free_s = free_b[used[1]:], free_s[used[2]:]
        at = 0
        for b, n in enumerate(step):
            outs[b].append((y[at:at + n], out[at:at + n]))
            at, done[b] = at + n, done[b] + n
    # decode: one token each, request 1 paused
    step = [1, 0, 1, 1, 1]
    rows = [b for b, n in enumerate(step) if n]
    maps = jamba_ssm_batch_maps(_i32(step), table, _i32(free_b), slots, _i32(free_s),
                                ctx_lens=_i32(done), block_size=bs, max_tokens=requests)
    assert maps["counts"].tolist()[0] == 4
    x, g, z = mixer_inputs(torch.stack([tokens[b][done[b]] for b in range(requests)]))
    y = jamba_ssm_gated_state_update(cache, x, g, z=z, rate=rate,
                                     state_indices=maps["state_indices"])
    for b in rows:
        outs[b].append((y[b:b + 1], project(y[b:b + 1], w_out, s_out)))
        done[b] += 1
    assert jamba_ssm_serve_get_status() == 0
    # every block of every table is held once
    held = [v for r in table.tolist() for v in r if v >= 0]
    assert len(held) == len(set(held)) == sum(-(-n // bs) for n in done)
    for b in range(requests):
        x, g, z = mixer_inputs(tokens[b][:done[b]])
        ref = Reference(x[None], g[None], z[None], rate)
        y = torch.cat([v[0] for v in outs[b]])
        assert_within(y, ref.out, ref.e_out, f"request {b}")
        assert torch.equal(torch.cat([v[1] for v in outs[b]]), project(y, w_out, s_out))
        assert_within(cache[int(slots[b])], ref.h_final[0], ref.e_final[0], f"state {b}")


def test_status_without_a_device_index():
    from selective_state_space_26_b200 import jamba_ssm_gated_get_status
    _i32([0])  # a device
    for device in (None, "cuda", torch.device("cuda"), 0):
        assert jamba_ssm_serve_get_status(device=device) == 0
        assert jamba_ssm_gated_get_status(device=device) == 0


def test_recycled_slots_and_the_selective_scan():
    """Two steps of a continuous batch through jamba_ssm_scan, then a decode step.  A
    request of the second step gets the slot of one that ended: its row was zeroed
    then, so every request's outputs are those of its tokens alone, from zero.  Left as
    it was, the row would be the new request's initial state."""
    from selective_state_space_26_b200 import (jamba_ssm_get_status, jamba_ssm_scan,
                                               jamba_ssm_state_update, synth)
    from tests.parity import assert_out
    from tests.test_gpu_serving import _oracle_seq
    _i32([0])
    d, n, bf = 128, 16, torch.bfloat16
    # rows: requests 0 to 3; request 3 comes in the second step
    inp = synth.scan_inputs(4, 90, d, n, bf, seed=21, device="cuda", A_kind="random")
    cache = torch.zeros(3, d, n, device="cuda")
    args = dict(D=inp.D, delta_bias=inp.delta_bias)
    done, free_s = [0] * 4, [2, 0, 1]
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    slots = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    outs = [[] for _ in range(4)]

    def step(who, lens):
        nonlocal free_s
        cat = lambda t: torch.cat([t[r, done[r]:done[r] + k] for r, k in zip(who, lens)])  # noqa: E731
        maps = jamba_ssm_batch_maps(_i32(lens), table, _i32(list(range(40))), slots, _i32(free_s),
                                    ctx_lens=_i32([done[r] for r in who]), block_size=16,
                                    max_tokens=sum(lens))
        free_s = free_s[maps["counts"].tolist()[2]:]
        out, _ = jamba_ssm_scan(cat(inp.x), cat(inp.delta), cat(inp.z), cat(inp.B), cat(inp.C),
                                inp.A, **args, h0=cache, h_final=cache,
                                cu_seqlens=maps["cu_seqlens"],
                                state_indices=maps["state_indices"])
        for r, k, o in zip(who, lens, out.split(lens)):
            outs[r].append(o)
            done[r] += k
        return maps

    step([0, 1, 2], [40, 17, 64])
    ended = int(slots[1])
    left = cache[ended].clone()
    assert left.abs().max() > 0
    cache[ended] = 0
    free_s.append(ended)
    table[1], slots[1] = -1, -1
    maps = step([0, 3, 2], [1, 50, 20])  # request 3 in the place of 1, with its slot
    assert maps["state_indices"].tolist()[1] == ended and maps["initial_indices"].tolist()[1] == -1
    maps = jamba_ssm_batch_maps(_i32([1, 1, 1]), table, _i32([]), slots, _i32([]),
                                ctx_lens=_i32([done[0], done[3], done[2]]), block_size=128,
                                max_tokens=3)
    row = lambda t: torch.stack([t[r, done[r]] for r in (0, 3, 2)])  # noqa: E731
    y = jamba_ssm_state_update(cache, row(inp.x), row(inp.delta), row(inp.z), row(inp.B),
                               row(inp.C), inp.A, **args, state_indices=maps["state_indices"])
    for i, r in enumerate((0, 3, 2)):
        outs[r].append(y[i:i + 1])
        done[r] += 1
    for r in range(4):
        ref, _ = _oracle_seq(inp, r, done[r])
        assert_out(torch.cat(outs[r]), ref, bf, f"request {r}")
    # the row left as it was
    stale = jamba_ssm_scan(inp.x[3, :50], inp.delta[3, :50], inp.z[3, :50], inp.B[3, :50],
                           inp.C[3, :50], inp.A, **args, h0=left[None], cu_seqlens=_i32([0, 50]),
                           h_final=left.clone()[None], state_indices=_i32([0]))[0]
    assert not torch.equal(stale, outs[3][0])
    assert jamba_ssm_get_status() == 0 and jamba_ssm_serve_get_status() == 0
