"""Cases of the operators beside the selective scan, and their plain forms.

The gated linear recurrence (forward, training step, one decode step), the int8
product with a scale for each token and each output channel, and the maps of a
continuous batch:

  scan   u = rate * sigmoid(g + bias),  h_t = h_{t-1} + u_t (x_t - h_{t-1}),
         out_t = h_t * silu(z_t)                       (without z: out_t = h_t)
  train  the scan and the gradients of every input from dout and dL/dh_final
  step   one token of the scan for each request, the state updated in place
  i8     q = round(x / s), s = max|x| / 127 for each token;
         out = (q . w_q) * s * s_w + bias
  maps   cu_seqlens, positions, block tables, cache slots and state slots of a
         batch from its requests' lengths

``own`` chooses between the plain forms (torch operations in 32 bits) and the
calls of selective_state_space_26_b200.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one 4096-token prompt through a layer of 8192 channels
        dict(name="scan_prefill", op="scan", packed=False, batch=1, tokens=4096, d=8192,
             dtype="bf16", gate=True),
        # prompts of one scheduler step, packed, read from one fused projection's output,
        # states in cache slots, some of them continued from an earlier chunk
        dict(name="scan_packed", op="scan", packed=True, batch=33, tokens=16384, d=4096,
             dtype="bf16", gate=True),
        # one long document in fp32, a width that no vector load divides, no output gate
        dict(name="scan_long", op="scan", packed=False, batch=1, tokens=50001, d=1001,
             dtype="f32", gate=False),
        # a training step's share of one layer: two sequences
        dict(name="train_layer", op="train", packed=False, batch=2, tokens=8192, d=4096,
             dtype="bf16", gate=True),
        # documents packed to one row, fp32
        dict(name="train_packed", op="train", packed=True, batch=9, tokens=3001, d=1000,
             dtype="f32", gate=True),
        # decode: one token for each of 256 requests of a 320-slot cache
        dict(name="step_batch", op="step", batch=256, d=8192, dtype="bf16", gate=True),
        # decode with few requests
        dict(name="step_few", op="step", batch=5, d=1027, dtype="f32", gate=False),
        # the layer's input projection (x | z, expansion 2) over a prompt
        dict(name="i8_prefill", op="i8", m=4096, k=4096, n=16384, dtype="bf16", bias=False),
        # the output projection in a decode step
        dict(name="i8_decode", op="i8", m=8, k=8192, n=4096, dtype="bf16", bias=False),
        # ragged sizes, a bias, fp32 in and out
        dict(name="i8_odd", op="i8", m=777, k=2050, n=1001, dtype="f32", bias=True),
        # a decode step's maps
        dict(name="maps_decode", op="maps", batch=256, tokens=256, block=16),
        # a step that mixes long prompts and decodes
        dict(name="maps_mixed", op="maps", batch=1000, tokens=131072, block=64),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("scan", "scan", "train", "train", "step", "i8", "i8", "maps"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("scan", "train"):
        packed = rng.random() < 0.5
        d = _between(rng, 33, 8192)
        if rng.random() < 0.6:
            d = -(-d // 8) * 8
        most = (1 << 25) if op == "scan" else (1 << 24)
        tokens = _between(rng, 1, min(65536, most // d))
        batch = _between(rng, 1, min(64, tokens))
        if not packed:
            tokens = max(1, tokens // batch) * batch
        return dict(op=op, packed=packed, batch=batch, tokens=tokens, d=d, dtype=dtype,
                    gate=rng.random() < 0.7)
    if op == "step":
        return dict(op=op, batch=_between(rng, 1, 256), d=_between(rng, 33, 8192), dtype=dtype,
                    gate=rng.random() < 0.7)
    if op == "i8":
        m, k, n = _between(rng, 1, 4096), _between(rng, 64, 8192), _between(rng, 64, 8192)
        if rng.random() < 0.5:
            k, n = -(-k // 128) * 128, -(-n // 128) * 128
        return dict(op=op, m=m, k=k, n=n, dtype=dtype, bias=rng.random() < 0.5)
    batch = _between(rng, 1, 1000)
    return dict(op=op, batch=batch, tokens=batch * _between(rng, 1, 128),
                block=rng.choice((16, 32, 64, 100)))


def work(case):
    c = case
    if c["op"] in ("scan", "train"):
        e, es = c["tokens"] * c["d"], BYTES[c["dtype"]]
        state = c["batch"] * c["d"] * 4
        arrays = 4 if c["gate"] else 3  # x, g, (z), out
        if c["op"] == "scan":
            return {"bytes": arrays * e * es + 2 * state, "flops": 12 * e}
        # the forward's, and x, g, (z), dout read and dx, dg, (dz) written
        back = 7 if c["gate"] else 5
        return {"bytes": (arrays + back) * e * es + 4 * state, "flops": 45 * e}
    if c["op"] == "step":
        e, es = c["batch"] * c["d"], BYTES[c["dtype"]]
        return {"bytes": e * ((4 if c["gate"] else 3) * es + 8), "flops": 12 * e}
    if c["op"] == "i8":
        es = BYTES[c["dtype"]]
        m, k, n = c["m"], c["k"], c["n"]
        return {"bytes": m * k * es + n * k + m * n * es + 4 * (m + n), "flops": 2 * m * n * k}
    # the lengths and free lists read, the per-token maps and the tables' new entries written
    return {"bytes": c["tokens"] * 16 + c["batch"] * 24 + 8 * (c["tokens"] // c["block"]),
            "flops": 8 * c["tokens"]}


# ------------------------------------------------------------------ inputs
def _randn(gen, dtype, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _lengths(rng, parts, total):
    """`total` cut into `parts` lengths, ragged; where there are more than three, the second is empty and the third is one."""
    if parts == 1:
        return [total]
    cuts = sorted(rng.randint(0, total) for _ in range(parts - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if parts > 3:
        last = max(range(3, parts), key=lambda i: lens[i])
        lens[last] += lens[1] + lens[2]
        lens[1], lens[2] = 0, 0
        if lens[last]:
            lens[last], lens[2] = lens[last] - 1, 1
    return lens


def prepare(case, seed):
    c = dict(case)
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["op"] in ("scan", "train", "step"):
        dt, d = DTYPES[c["dtype"]], c["d"]
        # a channel's memory: its rate cap is log-uniform in [1/300, 1]
        s["rate"] = torch.exp(torch.rand(d, generator=gen, device="cuda") * -math.log(300))
        s["bias"] = _randn(gen, torch.float32, d)
    if c["op"] in ("scan", "train"):
        t, b = c["tokens"], c["batch"]
        if c["packed"]:
            # x, g and z are column blocks of one projection's output, [tokens, 3 d]
            proj = _randn(gen, dt, t, (3 if c["gate"] else 2) * d)
            cols = proj.split(d, dim=1)
            s["x"], s["g"] = cols[0], cols[1]
            s["z"] = cols[2] if c["gate"] else None
            lens = _lengths(rng, b, t)
            s["cu"] = i32([sum(lens[:i]) for i in range(b + 1)])
        else:
            shape = (b, t // b, d)
            s["x"], s["g"] = _randn(gen, dt, *shape), _randn(gen, dt, *shape)
            s["z"] = _randn(gen, dt, *shape) if c["gate"] else None
            lens, s["cu"] = [t // b] * b, None
        s["lens"] = lens
        if c["op"] == "scan" and c["packed"]:
            slots = b + b // 4 + 1
            s["cache"] = _randn(gen, torch.float32, slots, d, std=0.3)
            order = rng.sample(range(slots), b)
            s["slots"] = i32(order)
            # two of three continue from their slot's state, the others start from zero
            s["initial"] = i32([v if i % 3 else -1 for i, v in enumerate(order)])
        else:
            s["h0"] = _randn(gen, torch.float32, b, d, std=0.3)
        if c["op"] == "train":
            s["dout"] = _randn(gen, dt, *s["x"].shape)
            s["dh"] = _randn(gen, torch.float32, b, d)
        # the plain form's row numbers
        starts = [sum(lens[:i]) for i in range(b)]
        full = [i for i in range(b) if lens[i]]
        s["full"] = torch.tensor(full, device="cuda")
        s["first"] = torch.tensor([starts[i] for i in full], device="cuda")
        s["last"] = torch.tensor([starts[i] + lens[i] - 1 for i in full], device="cuda")
    elif c["op"] == "step":
        b = c["batch"]
        s["x"], s["g"] = _randn(gen, dt, b, d), _randn(gen, dt, b, d)
        s["z"] = _randn(gen, dt, b, d) if c["gate"] else None
        slots = b + b // 4 + 1
        s["cache"] = _randn(gen, torch.float32, slots, d, std=0.3)
        s["slots"] = i32(rng.sample(range(slots), b))
    elif c["op"] == "i8":
        m, k, n = c["m"], c["k"], c["n"]
        # activations whose tokens differ in size
        size = torch.exp(torch.randn(m, 1, generator=gen, device="cuda") * 0.5)
        s["x"] = (torch.randn(m, k, generator=gen, device="cuda") * size).to(DTYPES[c["dtype"]])
        # the weight as it is kept: int8 rows padded with zeros to a multiple of 16 columns
        kp = -(-k // 16) * 16
        w = torch.zeros(n, kp, dtype=torch.int8, device="cuda")
        w[:, :k] = torch.randint(-127, 128, (n, k), generator=gen, device="cuda").to(torch.int8)
        s["w"] = w
        s["ws"] = torch.exp(torch.randn(n, generator=gen, device="cuda") * 0.3) / (127 * k ** 0.5)
        s["b"] = _randn(gen, torch.float32, n) if c["bias"] else None
    else:
        b, t, bs = c["batch"], c["tokens"], c["block"]
        if t == b:
            new = [1] * b
        else:
            new = _lengths(rng, b, t)
        # requests of one token continue a context, longer ones mostly begin
        ctx = [rng.randint(1, 8192) if n <= 1 or rng.random() < 0.3 else 0 for n in new]
        had = [-(-v // bs) for v in ctx]
        width = -(-(8192 + min(t, 8192)) // bs)  # the longest request that the table can hold
        pool = sum(max(had[i], -(-(ctx[i] + new[i]) // bs)) for i in range(b)) + 64
        blocks = list(range(pool))
        rng.shuffle(blocks)
        table = [[-1] * width for _ in range(b)]
        for i in range(b):
            for j in range(had[i]):
                table[i][j] = blocks.pop()
        slots = list(range(2 * b))
        rng.shuffle(slots)
        s["req"] = i32([slots.pop() if v else -1 for v in ctx])
        s["new"], s["ctx"], s["table"] = i32(new), i32(ctx), i32(table)
        s["free"], s["free_slots"] = i32(blocks), i32(slots)
        s["rows"] = t + 64  # the captured step's capacity: rows behind the batch are padding
    return s


# ------------------------------------------------------------- plain forms
def _recur(f, b, longest):
    """h_t = f_t h_{t-1} + b_t along the rows, where f is 0 at each sequence's first row: in ceil(log2 longest) rounds, each doubling the rows a value covers."""
    k = 1
    while k < longest:
        b = torch.cat((b[:k], torch.addcmul(b[k:], f[k:], b[:-k])))
        f = torch.cat((f[:k], f[k:] * f[:-k]))
        k *= 2
    return b


def _plain_scan(s):
    """(out, h_final, what the gradients need) in fp32."""
    c, d = s["case"], s["case"]["d"]
    x, g = s["x"].float().reshape(-1, d), s["g"].float().reshape(-1, d)
    sg = torch.sigmoid(g + s["bias"])
    u = s["rate"] * sg
    if c["op"] == "scan" and c["packed"]:
        at = s["initial"].long()
        h0 = torch.where((at >= 0)[:, None], s["cache"][at.clamp(min=0)], 0.0)
    else:
        h0 = s["h0"]
    f, b = 1 - u, u * x
    b[s["first"]] += f[s["first"]] * h0[s["full"]]
    f[s["first"]] = 0
    h = _recur(f, b, max(s["lens"]))
    hf = h0.clone()
    hf[s["full"]] = h[s["last"]]
    if s["z"] is not None:
        z = s["z"].float().reshape(-1, d)
        sz = torch.sigmoid(z)
        out = h * (z * sz)
    else:
        z = sz = None
        out = h
    return out, hf, (x, u, sg, h, h0, z, sz)


def _plain_grads(s, kept):
    x, u, sg, h, h0, z, sz = kept
    d = s["case"]["d"]
    dout = s["dout"].float().reshape(-1, d)
    dy = dout if z is None else dout * (z * sz)
    # g_t = dy_t + (1 - u_{t+1}) g_{t+1}, the recurrence with its rows reversed
    f = torch.cat((1 - u[1:], torch.zeros_like(u[:1])))
    dy = dy.clone()
    dy[s["last"]] += s["dh"][s["full"]]
    f[s["last"]] = 0
    gh = _recur(f.flip(0), dy.flip(0), max(s["lens"])).flip(0)
    before = torch.cat((h[:1], h[:-1]))
    before[s["first"]] = h0[s["full"]]
    du = gh * (x - before)
    dg = du * u * (1 - sg)
    dh0 = s["dh"].clone()
    dh0[s["full"]] = ((1 - u) * gh)[s["first"]]
    return {"dx": u * gh, "dg": dg,
            "dz": None if z is None else dout * h * (sz * (1 + z * (1 - sz))),
            "drate": (du * sg).sum(0, dtype=torch.float64).float(),
            "dbias": dg.sum(0, dtype=torch.float64).float(), "dh0": dh0}


def _plain_step(s):
    x, g, at = s["x"].float(), s["g"].float(), s["slots"].long()
    h = s["cache"][at]
    h = h + s["rate"] * torch.sigmoid(g + s["bias"]) * (x - h)
    s["cache"][at] = h
    out = h
    if s["z"] is not None:
        z = s["z"].float()
        out = h * (z * torch.sigmoid(z))
    return out.to(s["x"].dtype), s["cache"]


def _plain_i8(s):
    c = s["case"]
    x = s["x"].double()  # a quotient next to a half is told apart in 64 bits
    scale = (x.abs().amax(1) / 127).float()
    q = torch.round(x / scale.double()[:, None]).clamp(-127, 127)
    q = torch.where(scale[:, None] > 0, q, 0.0).float()
    out = (q @ s["w"][:, :c["k"]].float().T) * scale[:, None] * s["ws"]
    if s["b"] is not None:
        out = out + s["b"]
    return out.to(DTYPES[c["dtype"]])


def _plain_maps(s):
    bs, rows = s["case"]["block"], s["rows"]
    new, ctx, table = s["new"].long(), s["ctx"].long(), s["table"]
    r, width = table.shape
    cu = torch.zeros(r + 1, dtype=torch.int64, device=new.device)
    cu[1:] = new.cumsum(0).clamp(max=rows)
    n = cu[1:] - cu[:-1]
    had = (ctx + bs - 1) // bs
    need = torch.where(n > 0, (ctx + n + bs - 1) // bs, had)
    taken = (need - had).cumsum(0)
    at = torch.arange(width, device=new.device)[None, :]
    pick = at - had[:, None] + (taken - (need - had))[:, None]
    fresh = (at >= had[:, None]) & (at < need[:, None])
    table.copy_(torch.where(fresh, s["free"][pick.clamp(0, s["free"].numel() - 1)], table))
    t = torch.arange(rows, device=new.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=r - 1)
    live = t < cu[-1]
    pos = ctx[b] + t - cu[b]
    block = table[b, (pos // bs).clamp(0, width - 1)].long()
    starts = (n > 0) & (ctx == 0)
    nth = starts.long().cumsum(0)
    slot = s["free_slots"][(nth - 1).clamp(0, s["free_slots"].numel() - 1)]
    s["req"].copy_(torch.where(starts, slot, s["req"]))
    minus = torch.full((), -1, dtype=torch.int32, device=new.device)
    return {"cu_seqlens": cu.int(), "positions": torch.where(live, pos, -1).int(),
            "token_request": torch.where(live, b, -1).int(),
            "slot_map": torch.where(live & (block >= 0), block * bs + pos % bs, -1),
            "block_tables": table, "request_slots": s["req"],
            "state_indices": torch.where(n > 0, s["req"], minus),
            "initial_indices": torch.where((n > 0) & (ctx > 0), s["req"], minus),
            "counts": torch.stack((cu[-1], taken[-1], nth[-1], n.max())).int()}


# --------------------------------------------------------------------- run
def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    if c["op"] == "scan":
        out, hf, _ = _plain_scan(s)
        out = out.to(s["x"].dtype).reshape(s["x"].shape)
        if c["packed"]:
            s["cache"][s["slots"].long()] = hf
            hf = s["cache"]
        return {"out": out, "h_final": hf}
    if c["op"] == "train":
        out, hf, kept = _plain_scan(s)
        grads = _plain_grads(s, kept)
        r = {"out": out, **{k: grads[k] for k in ("dx", "dg", "dz")}}
        r = {k: None if v is None else v.to(s["x"].dtype).reshape(s["x"].shape) for k, v in r.items()}
        return {**r, "h_final": hf, **{k: grads[k] for k in ("drate", "dbias", "dh0")}}
    if c["op"] == "step":
        out, cache = _plain_step(s)
        return {"out": out, "state": cache}
    if c["op"] == "i8":
        return {"out": _plain_i8(s)}
    return _plain_maps(s)


def _own(s, c):
    import selective_state_space_26_b200 as jssm
    if c["op"] == "scan":
        if c["packed"]:
            out, hf = jssm.jamba_ssm_gated_scan(
                s["x"], s["g"], z=s["z"], rate=s["rate"], bias=s["bias"], h0=s["cache"],
                h_final=s["cache"], cu_seqlens=s["cu"], state_indices=s["slots"],
                initial_indices=s["initial"])
        else:
            out, hf = jssm.jamba_ssm_gated_scan(s["x"], s["g"], z=s["z"], rate=s["rate"],
                                                bias=s["bias"], h0=s["h0"])
        return {"out": out, "h_final": hf}
    if c["op"] == "train":
        ckpt = jssm.jamba_ssm_gated_scan_ckpt(s["x"], cu_seqlens=s["cu"])
        out, hf = jssm.jamba_ssm_gated_scan(s["x"], s["g"], z=s["z"], rate=s["rate"],
                                            bias=s["bias"], h0=s["h0"], cu_seqlens=s["cu"],
                                            ckpt=ckpt)
        grads = jssm.jamba_ssm_gated_scan_bwd(s["x"], s["g"], s["dout"], z=s["z"], rate=s["rate"],
                                              bias=s["bias"], h0=s["h0"], dh_final=s["dh"],
                                              cu_seqlens=s["cu"], ckpt=ckpt)
        return {"out": out, "h_final": hf, **grads}
    if c["op"] == "step":
        out = jssm.jamba_ssm_gated_state_update(s["cache"], s["x"], s["g"], z=s["z"],
                                                rate=s["rate"], bias=s["bias"],
                                                state_indices=s["slots"])
        return {"out": out, "state": s["cache"]}
    if c["op"] == "i8":
        q, scale = jssm.jamba_ssm_i8_quant(s["x"])
        return {"out": jssm.jamba_ssm_i8_proj(q, scale, s["w"], s["ws"], bias=s["b"],
                                              out_dtype=s["x"].dtype)}
    return jssm.jamba_ssm_batch_maps(s["new"], s["table"], s["free"], s["req"], s["free_slots"],
                                     ctx_lens=s["ctx"], block_size=c["block"],
                                     max_tokens=s["rows"])


# ----------------------------------------------------- the definition, fp64
def _exact_states(s):
    """Step by step in time, every sequence at once; (u, sigmoid, h before each row, h, h_final)."""
    c, d = s["case"], s["case"]["d"]
    x, g = s["x"].double().reshape(-1, d), s["g"].double().reshape(-1, d)
    sg = 1 / (1 + torch.exp(-(g + s["bias"].double())))
    u = s["rate"].double() * sg
    lens = torch.tensor(s["lens"], device=x.device)
    start = lens.cumsum(0) - lens
    if "cache" in s:
        keep = (s["initial"] >= 0).double()[:, None]
        h = s["cache"].double()[s["initial"].long().clamp(min=0)] * keep
    else:
        h = s["h0"].double().clone()
    before, after = torch.empty_like(x), torch.empty_like(x)
    ragged = len(set(s["lens"])) > 1
    for t in range(max(s["lens"])):
        if ragged:
            on = [i for i, n in enumerate(s["lens"]) if n > t]
            on = torch.tensor(on, device=x.device)
            row = start[on] + t
            before[row] = h[on]
            h[on] = (1 - u[row]) * h[on] + u[row] * x[row]
            after[row] = h[on]
        else:
            ut, b, a = (v.view(len(lens), -1, d)[:, t] for v in (u, before, after))
            b.copy_(h)
            h = (1 - ut) * h + ut * x.view(len(lens), -1, d)[:, t]
            a.copy_(h)
    return x, u, sg, before, after, h


def exact(case, seed):
    c = case
    if c["op"] == "maps":
        return None  # whole numbers
    s = prepare(case, seed)
    if c["op"] == "i8":
        x, k = s["x"].double(), c["k"]
        scale = (x.abs().max(dim=1).values / 127).float().double()  # held in 32 bits
        q = (x / scale[:, None]).round()
        q[scale == 0] = 0
        out = torch.einsum("mk,nk->mn", q, s["w"][:, :k].double())
        out = out * scale[:, None] * s["ws"].double()[None, :]
        return {"out": out if s["b"] is None else out + s["b"].double()}
    if c["op"] == "step":
        at = s["slots"].long()
        cache = s["cache"].double()
        u = s["rate"].double() / (1 + torch.exp(-(s["g"].double() + s["bias"].double())))
        h = (1 - u) * cache[at] + u * s["x"].double()
        cache[at] = h
        z = None if s["z"] is None else s["z"].double()
        return {"out": h if z is None else h * z / (1 + torch.exp(-z)), "state": cache}
    if c["tokens"] * c["d"] > 1 << 26 or max(s["lens"]) > 60000:
        return None
    x, u, sg, before, h, hf = _exact_states(s)
    shape, d = s["x"].shape, c["d"]
    z = None if s["z"] is None else s["z"].double().reshape(-1, d)
    gate = 1.0 if z is None else z / (1 + torch.exp(-z))
    out = (h * gate).reshape(shape)
    if c["op"] == "scan":
        if c["packed"]:
            cache = s["cache"].double()
            cache[s["slots"].long()] = hf
            hf = cache
        return {"out": out, "h_final": hf}
    dout = s["dout"].double().reshape(-1, d)
    lens = torch.tensor(s["lens"], device=x.device)
    start = lens.cumsum(0) - lens
    gh, gs = s["dh"].double().clone(), torch.empty_like(x)  # dL/dh_t
    dy = dout * gate
    for t in range(max(s["lens"]) - 1, -1, -1):
        on = torch.tensor([i for i, n in enumerate(s["lens"]) if n > t], device=x.device)
        row = start[on] + t
        now = gh[on] + dy[row]
        gs[row] = now
        gh[on] = now * (1 - u[row])
    du = gs * (x - before)
    dg = du * s["rate"].double() * sg * (1 - sg)
    dz = None
    if z is not None:
        sz = 1 / (1 + torch.exp(-z))
        dz = (dout * h * (sz + z * sz * (1 - sz))).reshape(shape)
    return {"out": out, "h_final": hf, "dx": (gs * u).reshape(shape), "dg": dg.reshape(shape),
            "dz": dz, "drate": (du * sg).sum(0), "dbias": dg.sum(0), "dh0": gh}
