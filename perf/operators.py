"""The operators around the SSD scan, as cases that can be timed and compared.

Three families, each in every direction that a Mamba-2 layer uses:

  conv       the short causal convolution that makes x, B and C from the
             projection: over whole prompts (conv_fwd, conv_bwd), and one
             token per sequence (conv_step)
  ssd_step   the single-token form of the scan: one state update and output
             per sequence, in place in a cache of states
  block_norm the norm after a block with its gate and residual scale, the
             residual sum, and the norm before the next block (block_norm_fwd,
             block_norm_bwd)

`own` chooses between the library's kernels and the plain form, which spells
the same formulas out in elementary torch operations in fp32.  `exact` gives
the results in fp64 in a third form: a sum of shifted copies, one head after
another, torch's rms_norm, and autograd for the gradients.
"""
import math

import torch
import torch.nn.functional as F

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _conv(name, op, lens, nx, nb, nc, width, dtype, packed=False, pad=0, init=False, final=False,
          act="silu", bias=True):
    """lens: "7" or "300,1,599" (packed) or "2x4096" (rows x tokens).  pad:
    channels of the projection's row that are not the convolution's (its row
    stride is nx + nb + nc + pad)."""
    return dict(name=name, op=op, lens=lens, nx=nx, nb=nb, nc=nc, width=width, dtype=dtype,
                packed=packed, pad=pad, init=init, final=final, act=act, bias=bias)


def _step(name, batch, nslots, heads, headdim, dstate, groups, dtype, padded=0, slots=True, pad=0):
    return dict(name=name, op="ssd_step", batch=batch, nslots=nslots, heads=heads, headdim=headdim,
                dstate=dstate, groups=groups, dtype=dtype, padded=padded, slots=slots, pad=pad)


def _cstep(name, batch, nslots, nx, nb, nc, width, dtype, padded=0, slots=True, pad=0):
    return dict(name=name, op="conv_step", batch=batch, nslots=nslots, nx=nx, nb=nb, nc=nc,
                width=width, dtype=dtype, padded=padded, slots=slots, pad=pad)


def _norm(name, op, tokens, channels, dtype, res, gate="none", post=False, scale=False, alpha=1.0):
    return dict(name=name, op=op, tokens=tokens, channels=channels, dtype=dtype, res=res, gate=gate,
                post=post, scale=scale, alpha=alpha)


def listed():
    return [
        # a short turn of a conversation that goes on from a cached state
        _conv("conv_fwd short turn", "conv_fwd", "1x17", 1536, 128, 128, 4, "bf16", pad=1560,
              init=True, final=True),
        # the training batch's layer: 64 heads of 64, 8 groups of 128
        _conv("conv_fwd training batch", "conv_fwd", "4x8192", 4096, 1024, 1024, 4, "bf16"),
        # the layer shape in training, read out of the projection's rows
        _conv("conv_bwd layer", "conv_bwd", "2x4096", 1536, 128, 128, 4, "bf16", pad=1560),
        # a packed batch of ragged sequences, one empty, in fp32
        _conv("conv_bwd packed ragged", "conv_bwd", "700,1,2,0,3070,64,513,1999", 128, 16, 16, 3,
              "f32", packed=True, init=True, final=True),
        # one conversation, one token
        _cstep("conv_step one row", 1, 1, 1536, 128, 128, 4, "bf16", slots=False, pad=1560),
        # a serving batch over a cache of slots, five rows of it padding
        _cstep("conv_step batch", 256, 300, 2048, 128, 128, 4, "bf16", padded=5),
        _step("ssd_step one row", 1, 1, 24, 64, 128, 1, "bf16", slots=False, pad=1816),
        _step("ssd_step batch", 256, 300, 32, 64, 128, 1, "bf16", padded=5),
        # one decoding step of a few conversations, fp32 residual stream
        _norm("block_norm_fwd decode", "block_norm_fwd", 4, 768, "bf16", "f32"),
        # a training batch's rows with every part in use
        _norm("block_norm_fwd batch", "block_norm_fwd", 32768, 2048, "bf16", "bf16", gate="silu",
              post=True, scale=True, alpha=0.22),
        _norm("block_norm_bwd layer", "block_norm_bwd", 8192, 768, "bf16", "f32", gate="sigmoid",
              post=True, scale=True),
        # an odd width and row count in fp32, the plain residual and norm
        _norm("block_norm_bwd odd", "block_norm_bwd", 5003, 1025, "f32", "f32", alpha=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_channels(rng, most):
    """(nx, nb, nc): heads x headdim and groups x dstate, or odd counts."""
    while True:
        if rng.random() < 0.75:
            groups = rng.choice((1, 2, 4, 8))
            nx = groups * rng.randint(1, 8) * rng.choice((16, 32, 64, 128))
            nb = nc = groups * rng.choice((16, 32, 64, 128))
        elif rng.random() < 0.5:
            nx, nb, nc = (_log_int(rng, 1, 700) for _ in range(3))
        else:
            nx, nb, nc = _log_int(rng, 1, 4000), 0, 0
        if nx + nb + nc <= most:
            return nx, nb, nc


def draw(rng):
    op = rng.choice(("conv_fwd", "conv_bwd", "conv_step", "ssd_step", "block_norm_fwd",
                     "block_norm_bwd"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("conv_fwd", "conv_bwd"):
        nx, nb, nc = _draw_channels(rng, 6144)
        most = max(1, min(32768, (40 if op == "conv_fwd" else 14) * 1000000 // (nx + nb + nc)))
        tokens = _log_int(rng, 1, most)
        packed = rng.random() < 0.4
        if packed:
            cuts = sorted(rng.randint(0, tokens) for _ in range(rng.randint(0, 40)))
            ends = cuts + [tokens]
            lens = ",".join(str(b - a) for a, b in zip([0] + cuts, ends))
        else:
            rows = rng.randint(1, min(8, tokens))
            lens = "%dx%d" % (rows, tokens // rows)
        c = _conv("", op, lens, nx, nb, nc, rng.randint(2, 4), dtype, packed,
                  rng.choice((0, 0, 8 * rng.randint(1, 200), rng.randint(1, 1000))),
                  rng.random() < 0.5, rng.random() < 0.5,
                  "silu" if rng.random() < 0.8 else "none", rng.random() < 0.8)
    elif op == "conv_step":
        nx, nb, nc = _draw_channels(rng, 6144)
        batch = _log_int(rng, 1, 300)
        slots = rng.random() < 0.7
        c = _cstep("", batch, batch + rng.randint(1, 60) if slots else batch, nx, nb, nc,
                   rng.randint(2, 4), dtype, rng.randint(0, batch // 4) if slots else 0, slots,
                   rng.choice((0, 0, rng.randint(1, 2000))))
    elif op == "ssd_step":
        groups = rng.choice((1, 1, 2, 4, 8))
        heads = groups * rng.randint(1, 8)
        headdim = rng.choice((32, 64, 64, 128, rng.randint(1, 100)))
        dstate = rng.choice((16, 32, 64, 128, 128, 256, rng.randint(1, 256)))
        batch = _log_int(rng, 1, max(1, min(300, 64000000 // (heads * headdim * dstate))))
        slots = rng.random() < 0.7
        c = _step("", batch, batch + rng.randint(1, 60) if slots else batch, heads, headdim, dstate,
                  groups, dtype, rng.randint(0, batch // 4) if slots else 0, slots,
                  rng.choice((0, 0, rng.randint(1, 2000))))
    else:
        channels = rng.choice((256, 512, 768, 1024, 1536, 2048, 4096, _log_int(rng, 1, 4096)))
        tokens = _log_int(rng, 1, max(1, min(40000, 25000000 // channels)))
        c = _norm("", op, tokens, channels, dtype, rng.choice((dtype, "f32")),
                  rng.choice(("none", "linear", "sigmoid", "silu")), rng.random() < 0.5,
                  rng.random() < 0.5, rng.choice((1.0, 0.22, 0.5)))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lens(case):
    """(rows, tokens per row, sequence lengths)."""
    if case["packed"]:
        lens = [int(v) for v in case["lens"].split(",")]
        return 1, sum(lens), lens
    b, t = (int(v) for v in case["lens"].split("x"))
    return b, t, [t] * b


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def unif(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    def slots_of():
        """Row -> cache slot: all different, slot 0 kept free; -1 where the row is padding."""
        if not case["slots"]:
            return None
        s = torch.randperm(case["nslots"] - 1, generator=g, device="cuda")[:case["batch"]] + 1
        if case["padded"]:
            s[torch.randperm(case["batch"], generator=g, device="cuda")[:case["padded"]]] = -1
        return s.to(torch.int32)

    s = dict(case)
    op = case["op"]
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        nx, nb, nc, K = case["nx"], case["nb"], case["nc"], case["width"]
        C = nx + nb + nc
        s["splits"] = (nx, nb, nc)
        r = 1.0 / math.sqrt(K)
        s["weight"] = unif(C, K, lo=-r, hi=r)
        s["bias"] = unif(C, lo=-r, hi=r) if case.get("bias", True) else None
        if op == "conv_step":
            # a view into the projection's rows: the convolution's channels
            s["x"] = randn(case["batch"], C + case["pad"], dtype=dt)[:, case["pad"]:]
            s["state"] = randn(case["nslots"], K - 1, C, dtype=dt)
            s["slots"] = slots_of()
            s["out"] = [torch.zeros((case["batch"], n), dtype=dt, device="cuda")
                        for n in s["splits"]]
            return s
        b, T, lens = _lens(case)
        n = len(lens)
        s["x"] = randn(b, T, C + case["pad"], dtype=dt)[..., case["pad"]:]
        s["init"] = randn(n, K - 1, C, dtype=dt) if case["init"] else None
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
        if op == "conv_bwd":
            s["dout"] = [randn(b, T, m, dtype=dt) for m in s["splits"]]
            s["dfinal"] = randn(n, K - 1, C, dtype=dt) if case["final"] else None
        return s
    if op == "ssd_step":
        B, H, P, N, G = (case[k] for k in ("batch", "heads", "headdim", "dstate", "groups"))
        row = randn(B, H * P + 2 * G * N + case["pad"], dtype=dt)
        # x, B and C lie side by side in one row, as the convolution leaves them
        s["x"] = row[:, :H * P].unflatten(1, (H, P))
        s["B"] = row[:, H * P:H * P + G * N].unflatten(1, (G, N))
        s["C"] = row[:, H * P + G * N:H * P + 2 * G * N].unflatten(1, (G, N))
        s["dt"] = (randn(B, H) - 2.0).to(dt)
        s["dt_bias"] = torch.log(torch.expm1(unif(H, lo=1e-3, hi=1e-1)))
        s["A"] = -torch.exp(unif(H, hi=math.log(16.0)))
        s["D"] = randn(H)
        s["state"] = randn(case["nslots"], H, P, N, scale=0.3)
        s["slots"] = slots_of()
        s["out"] = torch.zeros((B, H, P), dtype=dt, device="cuda")
        return s
    T, C = case["tokens"], case["channels"]
    rdt = DT[case["res"]]
    s["x"] = randn(T, C, dtype=dt)
    s["residual"] = randn(T, C, scale=3.0, dtype=rdt)
    s["gate_in"] = randn(T, C, scale=2.0, dtype=dt) if case["gate"] != "none" else None
    s["post_w"] = 1.0 + randn(C, scale=0.1) if case["post"] else None
    s["scale_w"] = 1.0 + randn(C, scale=0.3) if case["scale"] else None
    s["pre_w"] = 1.0 + randn(C, scale=0.1)
    s["eps"] = 1e-5
    if op == "block_norm_bwd":
        s["dout"] = randn(T, C, dtype=dt)
        s["dres"] = randn(T, C, dtype=rdt)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from state_space_model_ssd_amd import binding as lib
    op = s["op"]
    if op == "conv_fwd":
        *out, final = lib.conv_fwd(s["x"], s["weight"], s["bias"], splits=s["splits"],
                                   initial_states=s["init"], cu_seqlens=s["cu"],
                                   activation=s["act"], return_final_states=s["final"])
        return tuple(out), final
    if op == "conv_bwd":
        g = lib.conv_bwd(s["x"], s["weight"], s["dout"], s["bias"], splits=s["splits"],
                         initial_states=s["init"], cu_seqlens=s["cu"], activation=s["act"],
                         dfinal_states=s["dfinal"])
        return {k: g[k] for k in ("x", "weight", "bias", "initial_states")}
    if op == "conv_step":
        lib.conv_step(s["x"], s["state"], s["weight"], s["bias"], splits=s["splits"],
                      slots=s["slots"], outs=s["out"])
        return s["out"], s["state"]
    if op == "ssd_step":
        lib.ssd_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"],
                     dt_bias=s["dt_bias"], slots=s["slots"], out=s["out"])
        return s["out"], s["state"]
    kw = dict(gate=s["gate_in"], gate_activation=s["gate"] if s["gate"] != "none" else "linear",
              post_weight=s["post_w"], scale=s["scale_w"], residual_scale=s["alpha"], eps=s["eps"])
    if op == "block_norm_fwd":
        return lib.block_norm_fwd(s["x"], s["residual"], s["pre_w"], **kw)
    g = lib.block_norm_bwd(s["x"], s["residual"], s["pre_w"], s["dout"], s["dres"], **kw)
    return {k: g[k] for k in ("x", "residual", "gate", "post_weight", "scale", "pre_weight")}


def _run_plain(s):
    op = s["op"]
    if op in ("conv_fwd", "conv_bwd"):
        return _plain_conv(s)
    if op == "conv_step":
        return _plain_conv_step(s)
    if op == "ssd_step":
        return _plain_ssd_step(s)
    return _plain_norm_fwd(s) if op == "block_norm_fwd" else _plain_norm_bwd(s)


def _conv_plan(s):
    """Per token: its sequence's first and one-past-last token and its index;
    per sequence: first and one-past-last token."""
    b, T, _ = s["x"].shape
    dev = s["x"].device
    t = torch.arange(b * T, device=dev)
    if s["cu"] is not None:
        cu = s["cu"].long()
        first, last = cu[:-1], cu[1:]
        seq = torch.searchsorted(cu, t, right=True) - 1
    else:
        first = torch.arange(b, device=dev) * T
        last = first + T
        seq = t // T
    return t, seq, first, last


def _plain_conv(s):
    x, K, w = s["x"], s["width"], s["weight"]
    b, T, C = x.shape
    M = b * T
    t, seq, first, last = _conv_plan(s)
    n = first.numel()
    k = torch.arange(K, device=x.device)[:, None]
    r = torch.arange(K - 1, device=x.device)[None, :]
    pos = t - first[seq]
    raw = x.reshape(M, C)
    states = s["init"].reshape(n * (K - 1), C) if s["init"] is not None \
        else torch.zeros((n * (K - 1), C), dtype=x.dtype, device=x.device)
    src = torch.cat([raw, states])
    # tap k of token t: the token K - 1 - k before it, or a row of the initial state
    win = src[torch.where(pos + k >= K - 1, t - (K - 1) + k, M + seq * (K - 1) + pos + k)].float()
    pre = (win * w.t()[:, None, :]).sum(0)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    sig = torch.sigmoid(pre)
    silu = s["act"] == "silu"
    if s["op"] == "conv_fwd":
        out = (pre * sig if silu else pre).to(x.dtype).reshape(b, T, C).split(s["splits"], -1)
        final = None
        if s["final"]:
            tok = last[:, None] - (K - 1) + r
            len_ = (last - first)[:, None]
            row = M + torch.arange(n, device=x.device)[:, None] * (K - 1) + len_ + r
            final = src[torch.where(tok >= first[:, None], tok, row)]
        return tuple(o.contiguous() for o in out), final
    dout = torch.cat(s["dout"], -1).reshape(M, C).float()
    dpre = dout * (sig * (1.0 + pre * (1.0 - sig))) if silu else dout
    zero = torch.zeros((1, C), device=x.device)
    dpad = torch.cat([dpre, zero])
    dx = (dpad[torch.where(t + k < last[seq], t + k, M)] * w.flip(1).t()[:, None, :]).sum(0)
    len_ = (last - first)[:, None, None]
    # row r of the initial state is tap k of the sequence's token r - k
    tok = r[..., None] - k[:, 0]
    ok = (tok >= 0) & (tok < len_)
    dinit = (dpad[torch.where(ok, first[:, None, None] + tok, M)] * w.t()).sum(2)
    if s["dfinal"] is not None:
        df = torch.cat([s["dfinal"].reshape(n * (K - 1), C).float(), zero])
        i = t - (last[seq] - (K - 1))
        dx = dx + df[torch.where(i >= 0, seq * (K - 1) + i, n * (K - 1))]
        i = r - (last - first)[:, None]
        at = torch.arange(n, device=x.device)[:, None] * (K - 1) + i
        dinit = dinit + df[torch.where(i >= 0, at, n * (K - 1))]
    return {"x": dx.to(x.dtype).reshape(b, T, C), "weight": (win * dpre).sum(1).t().contiguous(),
            "bias": dpre.sum(0) if s["bias"] is not None else None,
            "initial_states": dinit.to(x.dtype) if s["init"] is not None else None}


def _row_slots(s):
    """Each row's slot (padding points at the free slot 0) and whether it has one."""
    if s["slots"] is None:
        i = torch.arange(s["x"].shape[0], device=s["x"].device)
        return i, torch.ones_like(i, dtype=torch.bool)
    return s["slots"].long().clamp(min=0), s["slots"] >= 0


def _plain_conv_step(s):
    idx, keep = _row_slots(s)
    old = s["state"][idx]
    win = torch.cat([old, s["x"][:, None, :]], 1)
    pre = (win.float() * s["weight"].t()).sum(1) + s["bias"]
    y = (pre * torch.sigmoid(pre)).to(s["x"].dtype)
    s["state"].index_copy_(0, idx, torch.where(keep[:, None, None], win[:, 1:], old))
    out = [o.copy_(torch.where(keep[:, None], v, o))
           for o, v in zip(s["out"], y.split(s["splits"], -1))]
    return out, s["state"]


def _plain_ssd_step(s):
    idx, keep = _row_slots(s)
    H, G = s["heads"], s["groups"]
    old = s["state"][idx]
    u = s["dt"].float() + s["dt_bias"]
    delta = u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))
    decay = torch.exp(delta * s["A"])
    x = s["x"].float()
    Bh = s["B"].float().repeat_interleave(H // G, 1)
    Ch = s["C"].float().repeat_interleave(H // G, 1)
    new = old * decay[..., None, None] + (x * delta[..., None])[..., None] * Bh[:, :, None, :]
    y = (new * Ch[:, :, None, :]).sum(-1) + x * s["D"][:, None]
    s["state"].index_copy_(0, idx, torch.where(keep[:, None, None, None], new, old))
    out = s["out"]
    return out.copy_(torch.where(keep[:, None, None], y.to(out.dtype), out)), s["state"]


def _plain_gate(s):
    """The gate's factor and its derivative."""
    if s["gate_in"] is None:
        return 1.0, 0.0
    z = s["gate_in"].float()
    if s["gate"] == "linear":
        return z, 1.0
    sig = torch.sigmoid(z)
    if s["gate"] == "sigmoid":
        return sig, sig * (1.0 - sig)
    return z * sig, sig * (1.0 + z * (1.0 - sig))


def _plain_norm_parts(s):
    x = s["x"].float()
    r1 = m = None
    p = x
    if s["post_w"] is not None:
        r1 = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        m = x * r1
        p = m * s["post_w"]
    act, dact = _plain_gate(s)
    u = p * act
    f = s["alpha"] * s["scale_w"] if s["scale_w"] is not None else s["alpha"]
    h = s["residual"].float() + u * f
    r2 = torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"])
    return r1, m, p, act, dact, u, f, h, r2


def _plain_norm_fwd(s):
    h, r2 = _plain_norm_parts(s)[-2:]
    return (h * r2 * s["pre_w"]).to(s["x"].dtype), h.to(s["residual"].dtype)


def _plain_norm_bwd(s):
    r1, m, p, act, dact, u, f, h, r2 = _plain_norm_parts(s)
    do = s["dout"].float()
    n = h * r2
    dn = do * s["pre_w"]
    dh = r2 * (dn - n * (dn * n).mean(-1, keepdim=True)) + s["dres"].float()
    du = dh * f
    dp = du * act
    g = {"residual": dh.to(s["residual"].dtype), "pre_weight": (do * n).sum(0),
         "scale": None, "gate": None, "post_weight": None}
    if s["scale_w"] is not None:
        g["scale"] = (dh * u * s["alpha"]).sum(0)
    if s["gate_in"] is not None:
        g["gate"] = (du * p * dact).to(s["x"].dtype)
    if s["post_w"] is not None:
        g["post_weight"] = (dp * m).sum(0)
        dm = dp * s["post_w"]
        dp = r1 * (dm - m * (dm * m).mean(-1, keepdim=True))
    g["x"] = dp.to(s["x"].dtype)
    return g


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("conv"):
        C, K = case["nx"] + case["nb"] + case["nc"], case["width"]
        if op == "conv_step":
            rows = case["batch"] - case["padded"]
            return {"bytes": rows * C * e * 2 * K + 4 * C * (K + 1), "flops": rows * C * (2 * K + 5)}
        b, T, lens = _lens(case)
        M, st = b * T, len(lens) * (K - 1) * C * e
        if op == "conv_fwd":
            return {"bytes": 2 * M * C * e + 4 * C * (K + 1) + st * (case["init"] + case["final"]),
                    "flops": M * C * (2 * K + 5)}
        return {"bytes": 3 * M * C * e + 8 * C * (K + 1) + st * (2 * case["init"] + case["final"]),
                "flops": M * C * (6 * K + 10)}
    if op == "ssd_step":
        rows = case["batch"] - case["padded"]
        H, P, N, G = (case[k] for k in ("heads", "headdim", "dstate", "groups"))
        return {"bytes": rows * (8 * H * P * N + e * (2 * H * P + 2 * G * N + H)),
                "flops": rows * H * P * (5 * N + 4)}
    r = 2 if case["res"] == "bf16" else 4
    el = case["tokens"] * case["channels"]
    gated = case["gate"] != "none"
    vec = 4 * case["channels"] * (1 + case["post"] + case["scale"])
    if op == "block_norm_fwd":
        return {"bytes": el * (2 * e + e * gated + 2 * r) + vec, "flops": el * 12}
    return {"bytes": el * (3 * e + 2 * e * gated + 3 * r) + 2 * vec, "flops": el * 35}


# ---------------------------------------------------------------------------
# fp64, written apart from the plain form
# ---------------------------------------------------------------------------
def _conv64(x, w, bias, splits, state, act):
    """One sequence (tokens, C) behind its state (K - 1, C), in fp64: a sum of
    shifted copies."""
    full = torch.cat([state, x])
    n, K = x.shape[0], w.shape[1]
    y = sum(full[k:k + n] * w[:, k] for k in range(K))
    if bias is not None:
        y = y + bias
    return (F.silu(y) if act == "silu" else y).split(splits, -1), full[n:]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def d(v, grad=False):
        if v is None:
            return None
        v = v.double()
        return v.requires_grad_(True) if grad else v

    if op in ("conv_fwd", "conv_bwd"):
        bwd = op == "conv_bwd"
        b, T, lens = _lens(case)
        if b * T * s["x"].shape[2] > 4e8:
            return None
        K, C = case["width"], s["x"].shape[2]
        x, w, bias = d(s["x"].contiguous(), bwd), d(s["weight"], bwd), d(s["bias"], bwd)
        init = torch.zeros((len(lens), K - 1, C), dtype=torch.float64, device=x.device)
        init = d(s["init"] if s["init"] is not None else init, bwd)
        flat, at, outs, finals = x.reshape(b * T, C), 0, [], []
        for i, n in enumerate(lens):
            o, f = _conv64(flat[at:at + n], w, bias, case_splits(case), init[i], case["act"]) if n \
                else ([flat[at:at, :m] for m in case_splits(case)], init[i])
            outs.append(o)
            finals.append(f)
            at += n
        out = [torch.cat([o[j] for o in outs]).reshape(b, T, -1) for j in range(3)]
        final = torch.stack(finals)
        if not bwd:
            return tuple(out), final if case["final"] else None
        loss = sum((o * g.double()).sum() for o, g in zip(out, s["dout"]))
        if s["dfinal"] is not None:
            loss = loss + (final * s["dfinal"].double()).sum()
        loss.backward()
        return {"x": x.grad, "weight": w.grad, "bias": bias.grad if bias is not None else None,
                "initial_states": init.grad if s["init"] is not None else None}
    if op == "conv_step":
        state, outs = s["state"].double(), [o.double() for o in s["out"]]
        w, bias, x = s["weight"].double(), s["bias"].double(), s["x"].double()
        slots = s["slots"].tolist() if s["slots"] is not None else list(range(case["batch"]))
        rows = [i for i, v in enumerate(slots) if v >= 0]
        at = [slots[i] for i in rows]
        full = torch.cat([state[at], x[rows][:, None]], 1)
        y = F.silu(torch.einsum("bkc,ck->bc", full, w) + bias)
        state[at] = full[:, 1:]
        for o, v in zip(outs, y.split(case_splits(case), -1)):
            o[rows] = v
        return outs, state
    if op == "ssd_step":
        state, out = s["state"].double(), s["out"].double()
        slots = s["slots"].tolist() if s["slots"] is not None else list(range(case["batch"]))
        delta = F.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=700.0)
        hpg = case["heads"] // case["groups"]
        for h in range(case["heads"]):
            rows = [i for i, v in enumerate(slots) if v >= 0]
            at = [slots[i] for i in rows]
            dl = delta[rows, h]
            x, Bv, Cv = (s[k].double()[rows] for k in ("x", "B", "C"))
            new = state[at, h] * torch.exp(dl * s["A"].double()[h])[:, None, None]
            new = new + torch.einsum("b,bp,bn->bpn", dl, x[:, h], Bv[:, h // hpg])
            state[at, h] = new
            out[rows, h] = (new * Cv[:, h // hpg][:, None]).sum(-1) + s["D"].double()[h] * x[:, h]
        return out, state
    bwd = op == "block_norm_bwd"
    if case["tokens"] * case["channels"] > 1e8:
        return None
    x, res, gate = d(s["x"], bwd), d(s["residual"], bwd), d(s["gate_in"], bwd)
    post, sc, pre = d(s["post_w"], bwd), d(s["scale_w"], bwd), d(s["pre_w"], bwd)
    C = case["channels"]
    u = F.rms_norm(x, (C,), post, s["eps"]) if post is not None else x
    if gate is not None:
        u = u * {"linear": lambda v: v, "sigmoid": torch.sigmoid, "silu": F.silu}[case["gate"]](gate)
    u = u * case["alpha"]
    h = res + (u * sc if sc is not None else u)
    out = F.rms_norm(h, (C,), pre, s["eps"])
    if not bwd:
        return out, h
    ((out * s["dout"].double()).sum() + (h * s["dres"].double()).sum()).backward()
    of = lambda v: v.grad if v is not None else None  # noqa: E731
    return {"x": x.grad, "residual": res.grad, "gate": of(gate), "post_weight": of(post),
            "scale": of(sc), "pre_weight": pre.grad}


def case_splits(case):
    return case["nx"], case["nb"], case["nc"]
