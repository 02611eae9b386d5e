"""The operators of a gated delta layer, as cases that can be timed and compared.

Two families, each in every direction that such a layer uses:

  delta     the gated delta rule, S_t = a_t S_(t-1) + w_t k_t^T with
            w_t = beta_t (v_t - a_t S_(t-1) k_t), a_t = exp(g_t), and
            o_t = scale S_t q_t: over whole prompts (delta_fwd, delta_bwd), and
            one token per sequence, in place in a cache of states (delta_step)
  qk_norm   the norm of queries and keys in each head, and the rotation by the
            token's position, in one pass (qk_norm_fwd, qk_norm_bwd)

`own` chooses between the library's kernels and the plain form.  The plain form
of delta is the chunked one in fp32 (products of 64-token blocks, their
triangular systems by halves, one state per chunk); `exact` is the recurrence
itself, one token after another in fp64, and its gradients by hand.
"""
import math

import torch
import torch.nn.functional as F

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _delta(name, op, lens, heads, groups, headdim, dstate, dtype, packed=False, init=False,
           final=False):
    """lens: "7" or "300,1,599" (packed) or "2x4096" (rows x tokens)."""
    return dict(name=name, op=op, lens=lens, heads=heads, groups=groups, headdim=headdim,
                dstate=dstate, dtype=dtype, packed=packed, init=init, final=final)


def _step(name, batch, nslots, heads, groups, headdim, dstate, dtype, padded=0, slots=True, pad=0):
    return dict(name=name, op="delta_step", batch=batch, nslots=nslots, heads=heads, groups=groups,
                headdim=headdim, dstate=dstate, dtype=dtype, padded=padded, slots=slots, pad=pad)


def _norm(name, op, tokens, q_heads, k_heads, headdim, dtype, norm="rms", weights=True, rotary=0,
          interleaved=False, far=4096, pad=0):
    """rotary: channels of a head that are rotated; far: positions are below it;
    pad: channels of the projection's row that are neither queries nor keys."""
    return dict(name=name, op=op, tokens=tokens, q_heads=q_heads, k_heads=k_heads, headdim=headdim,
                dtype=dtype, norm=norm, weights=weights, rotary=rotary, interleaved=interleaved,
                far=far, pad=pad)


def listed():
    return [
        # a short turn of a conversation that goes on from a cached state
        _delta("delta_fwd short turn", "delta_fwd", "1x17", 32, 16, 128, 128, "bf16", init=True,
               final=True),
        # prompts of a serving batch, packed and ragged, one empty: their states go to the cache
        _delta("delta_fwd packed prompts", "delta_fwd", "700,1,2,0,2900,64,513,1999,8192", 24, 8,
               64, 128, "bf16", packed=True, final=True),
        # a training batch
        _delta("delta_fwd training batch", "delta_fwd", "4x8192", 32, 16, 128, 128, "bf16"),
        # one row of training
        _delta("delta_bwd layer", "delta_bwd", "2x4096", 32, 16, 128, 128, "bf16"),
        # segments of a packed batch that carry their states on, in fp32
        _delta("delta_bwd packed ragged", "delta_bwd", "700,1,2,0,1530,64,513", 8, 4, 64, 64, "f32",
               packed=True, init=True, final=True),
        # one conversation, one token
        _step("delta_step one row", 1, 1, 32, 16, 128, 128, "bf16", slots=False, pad=512),
        # a serving batch over a cache of slots, five rows of it padding
        _step("delta_step batch", 256, 300, 32, 16, 128, 128, "bf16", padded=5),
        # one decoding step of a few conversations, far into their texts
        _norm("qk_norm_fwd decode", "qk_norm_fwd", 4, 32, 8, 128, "bf16", rotary=128, far=500000,
              pad=1024),
        # the delta layer's own norm: a training batch, unit length, no weights
        _norm("qk_norm_fwd unit length", "qk_norm_fwd", 32768, 16, 16, 128, "bf16", norm="l2",
              weights=False),
        # an attention layer of a hybrid model in training, read out of the projection's rows
        _norm("qk_norm_bwd layer", "qk_norm_bwd", 8192, 32, 8, 128, "bf16", rotary=128, pad=1024),
        # odd counts in fp32, neighbouring channels as pairs, a part of each head rotated
        _norm("qk_norm_bwd odd", "qk_norm_bwd", 5003, 7, 3, 100, "f32", rotary=34,
              interleaved=True, far=100000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("delta_fwd", "delta_bwd", "delta_step", "qk_norm_fwd", "qk_norm_bwd"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("delta_fwd", "delta_bwd"):
        groups = rng.choice((1, 2, 3, 4, 8, 16))
        heads = groups * rng.choice((1, 1, 2, 4))
        headdim, dstate = rng.choice((16, 32, 64, 64, 128, 128, 192)), rng.choice((32, 64, 128, 128))
        # the largest listed ones: 4x8192 tokens of 32 heads of 128 x 128, a third of it backward;
        # fp32 has its own rate
        most = (4 if op == "delta_fwd" else 1) * 8192 * 32 * 128 * 128 // (8 if dtype == "f32" else 1)
        tokens = _log_int(rng, 1, max(1, min(16384, most // (heads * headdim * dstate))))
        packed = rng.random() < 0.5
        if packed:
            cuts = sorted(rng.randint(0, tokens) for _ in range(rng.randint(0, 20)))
            lens = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))
        else:
            rows = rng.randint(1, min(4, tokens))
            lens = "%dx%d" % (rows, tokens // rows)
        c = _delta("", op, lens, heads, groups, headdim, dstate, dtype, packed, rng.random() < 0.5,
                   rng.random() < 0.5)
    elif op == "delta_step":
        groups = rng.choice((1, 2, 4, 8, 16))
        heads = groups * rng.choice((1, 2, 4))
        headdim = rng.choice((32, 64, 128, 128, rng.randint(1, 100)))
        dstate = rng.choice((32, 64, 128, 128, 256, rng.randint(1, 256)))
        batch = _log_int(rng, 1, max(1, min(300, 128000000 // (heads * headdim * dstate))))
        slots = rng.random() < 0.7
        c = _step("", batch, batch + rng.randint(1, 60) if slots else batch, heads, groups, headdim,
                  dstate, dtype, rng.randint(0, batch // 4) if slots else 0, slots,
                  rng.choice((0, 0, rng.randint(1, 2000))))
    else:
        headdim = rng.choice((64, 128, 128, 256, rng.randint(2, 256)))
        q_heads, k_heads = rng.choice(((32, 8), (16, 16), (8, 1), (rng.randint(1, 40), rng.randint(1, 20))))
        rotary = rng.choice((0, headdim // 2 * 2, headdim // 4 * 2, 2 * rng.randint(1, headdim // 2)))
        tokens = _log_int(rng, 1, max(1, min(40000, 60000000 // (headdim * (q_heads + k_heads)))))
        c = _norm("", op, tokens, q_heads, k_heads, headdim, dtype, rng.choice(("rms", "l2")),
                  rng.random() < 0.7, rotary, rng.random() < 0.4, rng.choice((4096, 100000, 1000000)),
                  rng.choice((0, 8 * rng.randint(1, 200), rng.randint(1, 1000))))
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

    def heads_of(*shape, unit=True):
        """What a layer's convolution gives: SiLU of about normal values, queries and keys of
        unit length in each head."""
        x = F.silu(randn(*shape))
        return (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) if unit else x).to(dt)

    def gates(*lead):
        """Log decays A softplus(dt + bias) and step sizes: from heads that keep nearly
        everything to heads that forget in a few tokens."""
        H = case["heads"]
        bias = torch.log(torch.expm1(torch.exp(unif(H, lo=math.log(1e-3), hi=math.log(1e-1)))))
        decay = -unif(H, lo=0.1, hi=16.0) * F.softplus(randn(*lead, H) + bias)
        return decay.to(dt), torch.sigmoid(randn(*lead, H)).to(dt)

    s = dict(case)
    op = case["op"]
    if op in ("delta_fwd", "delta_bwd"):
        b, T, lens = _lens(case)
        H, G, P, N, n = (*(case[k] for k in ("heads", "groups", "headdim", "dstate")), len(lens))
        s["seqs"] = lens
        s["q"], s["k"] = heads_of(b, T, G, N), heads_of(b, T, G, N)
        s["v"] = heads_of(b, T, H, P, unit=False)
        s["g"], s["beta"] = gates(b, T)
        s["scale"] = N ** -0.5
        s["init"] = randn(n, H, P, N, scale=0.1) if case["init"] else None
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
        if op == "delta_bwd":
            s["dout"] = randn(b, T, H, P, dtype=dt)
            s["dfinal"] = randn(n, H, P, N) if case["final"] else None
        return s
    if op == "delta_step":
        B, H, G, P, N = (case[k] for k in ("batch", "heads", "groups", "headdim", "dstate"))
        # queries, keys and values lie side by side in one row, as the convolution leaves them
        row = F.silu(randn(B, 2 * G * N + H * P + case["pad"]))
        row[:, :2 * G * N].unflatten(1, (2 * G, N)).div_(
            row[:, :2 * G * N].unflatten(1, (2 * G, N)).norm(dim=-1, keepdim=True) + 1e-6)
        row = row.to(dt)
        s["q"] = row[:, :G * N].unflatten(1, (G, N))
        s["k"] = row[:, G * N:2 * G * N].unflatten(1, (G, N))
        s["v"] = row[:, 2 * G * N:2 * G * N + H * P].unflatten(1, (H, P))
        s["g"], s["beta"] = gates(B)
        s["scale"] = N ** -0.5
        s["state"] = randn(case["nslots"], H, P, N, scale=0.3)
        s["slots"] = None
        if case["slots"]:
            # all different, slot 0 kept free; -1 where the row is padding
            at = torch.randperm(case["nslots"] - 1, generator=g, device="cuda")[:B] + 1
            if case["padded"]:
                at[torch.randperm(B, generator=g, device="cuda")[:case["padded"]]] = -1
            s["slots"] = at.to(torch.int32)
        s["out"] = torch.zeros((B, H, P), dtype=dt, device="cuda")
        return s
    T, Hq, Hk, D = (case[k] for k in ("tokens", "q_heads", "k_heads", "headdim"))
    row = randn(T, (Hq + Hk) * D + case["pad"], scale=2.0, dtype=dt)
    s["q"] = row[:, :Hq * D].unflatten(1, (Hq, D))
    s["k"] = row[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    s["q_w"] = 1.0 + randn(D, scale=0.2) if case["weights"] else None
    s["k_w"] = 1.0 + randn(D, scale=0.2) if case["weights"] else None
    s["eps"] = 1e-6
    s["pos"] = s["freq"] = None
    if case["rotary"]:
        R = case["rotary"] // 2
        s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["freq"] = (10000.0 ** (-torch.arange(R, dtype=torch.float64) / R)).float().cuda()
    if op == "qk_norm_bwd":
        s["dq"], s["dk"] = randn(T, Hq, D, dtype=dt), randn(T, Hk, D, dtype=dt)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from state_space_model_ssd_amd import binding as lib
    op = s["op"]
    if op == "delta_fwd":
        out, final, _ = lib.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"],
                                      initial_states=s["init"], cu_seqlens=s["cu"],
                                      return_final_states=s["final"])
        return out, final
    if op == "delta_bwd":
        g = lib.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], scale=s["scale"],
                          initial_states=s["init"], cu_seqlens=s["cu"], dfinal_states=s["dfinal"])
        return {k: g[k] for k in ("q", "k", "v", "g", "beta", "initial_states")}
    if op == "delta_step":
        lib.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"],
                       slots=s["slots"], out=s["out"])
        return s["out"], s["state"]
    kw = dict(norm=s["norm"], eps=s["eps"], positions=s["pos"], inv_freq=s["freq"],
              interleaved=s["interleaved"])
    if op == "qk_norm_fwd":
        return lib.qk_norm_fwd(s["q"], s["k"], s["q_w"], s["k_w"], **kw)
    g = lib.qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], s["q_w"], s["k_w"], **kw)
    return {k: g[k] for k in ("q", "k", "q_weight", "k_weight")}


def _run_plain(s):
    op = s["op"]
    if op == "delta_fwd":
        return _plain_delta_fwd(s)
    if op == "delta_bwd":
        return _plain_delta_bwd(s)
    if op == "delta_step":
        return _plain_delta_step(s)
    return _plain_qk_norm(s)


def _chunk_index(s):
    """Token of (sequence, chunk, row), the number of tokens where there is none; and where each
    token lies in that table."""
    dev, n = s["q"].device, len(s["seqs"])
    M = s["q"].shape[0] * s["q"].shape[1]
    chunks = max(1, -(-max(s["seqs"], default=0) // CHUNK))
    at = torch.arange(chunks * CHUNK, device=dev)
    if s["cu"] is not None:
        cu = s["cu"].long()
        first, last = cu[:-1], cu[1:]
    else:
        first = torch.arange(n, device=dev) * s["q"].shape[1]
        last = first + s["q"].shape[1]
    tok = first[:, None] + at
    tok = torch.where(tok < last[:, None], tok, M)
    back = torch.zeros(M + 1, dtype=torch.long, device=dev)
    back[tok.flatten()] = torch.arange(tok.numel(), device=dev)
    return tok.reshape(n, chunks, CHUNK), back[:M]


def _chunked(x, tok, repeat=1):
    """(b, T, heads, ...) -> fp32 (sequences, chunks, heads * repeat, CHUNK, ...), zeros where
    there is no token."""
    x = x.flatten(0, 1).float()
    x = torch.cat([x, torch.zeros_like(x[:1])])[tok].transpose(2, 3)
    return x.repeat_interleave(repeat, 2) if repeat > 1 else x


def _lower(x, diagonal=0):
    return torch.tril(x, diagonal)


def _delta_parts(s, tok):
    """What does not depend on the state: per sequence, chunk and head."""
    rep = s["heads"] // s["groups"]
    q, k = _chunked(s["q"], tok, rep), _chunked(s["k"], tok, rep)
    v, beta = _chunked(s["v"], tok), _chunked(s["beta"], tok)[..., None]
    # the running sum of up to 64 log decays, whose small differences count, in 64 bits
    G = _chunked(s["g"], tok).double().cumsum(-1)
    q = q * s["scale"]
    E = torch.exp(G).float()[..., None]
    D = torch.exp(_lower(G[..., :, None] - G[..., None, :])).float()
    Dc = torch.exp(G[..., -1:] - G).float()[..., None]
    kt = k.transpose(-1, -2).contiguous()
    L = _lower(beta * D * (k @ kt), -1)
    # (1 + L)^-1 by halves: two inverted blocks of n rows and what couples them give one of 2 n
    row = torch.arange(CHUNK, device=L.device)
    inv = torch.eye(CHUNK, device=L.device).expand_as(L)
    for n in (1, 2, 4, 8, 16, 32):
        pair = (row[:, None] // (2 * n) == row // (2 * n)) & (row[:, None] // n != row // n)
        inv = inv - inv @ (torch.where(pair, L, 0.0) @ inv)
    A = _lower(D * (q @ kt))
    return q, k, v, beta, E, D, Dc, inv, A, inv @ (beta * v), inv @ (beta * E * k), L


def _plain_states(s, parts):
    """States entering each chunk, the state at the end, and the rows W = U - Wk S^T."""
    _, k, _, _, E, _, Dc, _, _, U, Wk, _ = parts
    n, chunks, H = U.shape[:3]
    S = s["init"] if s["init"] is not None else U.new_zeros(n, H, s["headdim"], s["dstate"])
    into, rows = [], []
    for c in range(chunks):
        into.append(S)
        W = U[:, c] - Wk[:, c] @ S.transpose(-1, -2).contiguous()
        rows.append(W)
        S = E[:, c, :, -1:] * S + (Dc[:, c] * W).transpose(-1, -2).contiguous() @ k[:, c]
    return torch.stack(into, 1), S, torch.stack(rows, 1)


def _unchunked(x, back, shape, dtype):
    """The inverse of _chunked: (sequences, chunks, heads, CHUNK, ...) -> (b, T, heads, ...)."""
    return x.transpose(2, 3).flatten(0, 2)[back].reshape(shape).to(dtype)


def _plain_delta_fwd(s):
    tok, back = _chunk_index(s)
    parts = _delta_parts(s, tok)
    q, E, A = parts[0], parts[4], parts[8]
    S, last, W = _plain_states(s, parts)
    o = E * (q @ S.transpose(-1, -2).contiguous()) + A @ W
    return _unchunked(o, back, s["v"].shape, s["v"].dtype), last if s["final"] else None


def _plain_delta_bwd(s):
    tok, back = _chunk_index(s)
    parts = _delta_parts(s, tok)
    q, k, v, beta, E, D, Dc, inv, A, _, Wk, L = parts
    S, _, W = _plain_states(s, parts)
    do = _chunked(s["dout"], tok)

    def t(x):
        return x.transpose(-1, -2).contiguous()

    Qh = E * q - A @ Wk
    dS = s["dfinal"] if s["dfinal"] is not None else torch.zeros_like(S[:, 0])
    leave = []
    for c in reversed(range(S.shape[1])):
        leave.append(dS)
        Z = Dc[:, c] * (k[:, c] @ t(dS))
        dS = E[:, c, :, -1:] * dS + t(do[:, c]) @ Qh[:, c] - t(Z) @ Wk[:, c]
    dSc = torch.stack(leave[::-1], 1)
    dR = t(inv) @ (t(A) @ do + Dc * (k @ t(dSc)))
    dL, dA = -_lower(dR @ t(W), -1), _lower(do @ t(W))
    # the decays between token j and a later token i are those of the tokens after j up to i
    pair = _lower(dA * A, -1) + dL * L
    dL, dA = dL * D, dA * D
    read, inter = E * (dR @ S), E * (do @ S)
    X = dL @ k - read
    dq = inter + dA @ k
    dk_in = beta * X
    state = Dc * (W @ dSc)
    dk_out = t(dA) @ q + state + t(beta * dL) @ k
    left = (q * inter - beta * k * read).sum(-1).double()
    kept = (k * state).sum(-1).double()
    pair = pair.double()
    dg = left.flip(-1).cumsum(-1).flip(-1) + (E[..., -1, 0] * (dSc * S).sum((-1, -2))).double()[..., None]
    dg = (dg + F.pad((kept + pair.sum(-2) - pair.sum(-1)).cumsum(-1), (1, -1))).float()
    dbeta = (dR * v).sum(-1) + (k * X).sum(-1)

    def grouped(x):
        return x.unflatten(2, (s["groups"], -1)).sum(3)

    return {"q": _unchunked(grouped(dq * s["scale"]), back, s["q"].shape, s["q"].dtype),
            "k": _unchunked(grouped(dk_in + dk_out), back, s["k"].shape, s["k"].dtype),
            "v": _unchunked(beta * dR, back, s["v"].shape, s["v"].dtype),
            "g": _unchunked(dg, back, s["g"].shape, s["g"].dtype),
            "beta": _unchunked(dbeta, back, s["beta"].shape, s["beta"].dtype),
            "initial_states": dS if s["init"] is not None else None}


def _plain_delta_step(s):
    B, rep = s["q"].shape[0], s["heads"] // s["groups"]
    if s["slots"] is None:
        idx = torch.arange(B, device=s["q"].device)
        keep = torch.ones_like(idx, dtype=torch.bool)
    else:
        idx, keep = s["slots"].long().clamp(min=0), s["slots"] >= 0
    old = s["state"][idx]
    q = s["q"].float().repeat_interleave(rep, 1)[:, :, None] * s["scale"]
    k = s["k"].float().repeat_interleave(rep, 1)[:, :, None]
    a = torch.exp(s["g"].float())[..., None]
    w = s["beta"].float()[..., None] * (s["v"].float() - a * (old * k).sum(-1))
    new = a[..., None] * old + w[..., None] * k
    y = (new * q).sum(-1).to(s["out"].dtype)
    s["state"].index_copy_(0, idx, torch.where(keep[:, None, None, None], new, old))
    return s["out"].copy_(torch.where(keep[:, None, None], y, s["out"])), s["state"]


def _angles(s):
    """cos and sin of position times frequency, by turns in fp64: far positions are many turns."""
    turns = s["pos"].double()[:, None] * s["freq"].double() / (2 * math.pi)
    a = ((turns - torch.floor(turns)) * (2 * math.pi)).float()
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def _rotated(x, s, cos, sin):
    """The first channels of each head turned by (cos, sin), in pairs."""
    R = cos.shape[-1]
    rot, rest = x[..., :2 * R], x[..., 2 * R:]
    if s["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :R], rot[..., R:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, rest], -1)


def _plain_qk_norm(s):
    cos = sin = None
    if s["pos"] is not None:
        cos, sin = _angles(s)
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s[name + "_w"]
        m = (x * x).mean(-1, keepdim=True) if s["norm"] == "rms" else (x * x).sum(-1, keepdim=True)
        r = torch.rsqrt(m + s["eps"])
        n = x * r
        if s["op"] == "qk_norm_fwd":
            y = n * w if w is not None else n
            out[name] = (_rotated(y, s, cos, sin) if cos is not None else y).to(s["q"].dtype)
            continue
        d = s["d" + name].float()
        if cos is not None:
            d = _rotated(d, s, cos, -sin)
        out[name + "_weight"] = (d * n).sum((0, 1)) if w is not None else None
        dn = d * w if w is not None else d
        dot = (dn * n).mean(-1, keepdim=True) if s["norm"] == "rms" else (dn * n).sum(-1, keepdim=True)
        out[name] = (r * (dn - n * dot)).to(s["q"].dtype)
    if s["op"] == "qk_norm_fwd":
        return out["q"], out["k"]
    return {k: out[k] for k in ("q", "k", "q_weight", "k_weight")}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("delta"):
        H, G, P, N = (case[k] for k in ("heads", "groups", "headdim", "dstate"))
        if op == "delta_step":
            rows = case["batch"] - case["padded"]
            return {"bytes": rows * (8 * H * P * N + e * 2 * (H * P + G * N + H)),
                    "flops": rows * H * P * (7 * N + 4)}
        b, T, lens = _lens(case)
        M, st = b * T, 4 * len(lens) * H * P * N
        row = 2 * G * N + H * P + 2 * H                     # q, k, v, g, beta
        if op == "delta_fwd":
            return {"bytes": M * e * (row + H * P) + st * (case["init"] + case["final"]),
                    "flops": M * H * P * N * 7}
        return {"bytes": M * e * (2 * row + H * P) + st * (2 * case["init"] + case["final"]),
                "flops": M * H * P * N * 22}
    T, D = case["tokens"], case["headdim"]
    el = T * D * (case["q_heads"] + case["k_heads"])
    rot = (4 * T + 2 * case["rotary"]) if case["rotary"] else 0
    w = 8 * D if case["weights"] else 0
    if op == "qk_norm_fwd":
        return {"bytes": 2 * e * el + w + rot, "flops": 8 * el}
    return {"bytes": 3 * e * el + 2 * w + rot, "flops": 16 * el}


# ---------------------------------------------------------------------------
# fp64, written apart from the plain form
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("delta_fwd", "delta_bwd"):
        return _exact_delta(case, s)
    if op == "delta_step":
        state, out = s["state"].double(), s["out"].double()
        slots = s["slots"].tolist() if s["slots"] is not None else list(range(case["batch"]))
        rows = [i for i, v in enumerate(slots) if v >= 0]
        at = [slots[i] for i in rows]
        hpg = case["heads"] // case["groups"]
        for h in range(case["heads"]):
            q, k = (s[n].double()[rows, h // hpg] for n in ("q", "k"))
            S = state[at, h] * torch.exp(s["g"].double()[rows, h])[:, None, None]
            w = s["beta"].double()[rows, h, None] * (s["v"].double()[rows, h]
                                                     - torch.einsum("bpn,bn->bp", S, k))
            S = S + torch.einsum("bp,bn->bpn", w, k)
            state[at, h] = S
            out[rows, h] = s["scale"] * torch.einsum("bpn,bn->bp", S, q)
        return out, state
    if case["tokens"] * case["headdim"] * (case["q_heads"] + case["k_heads"]) > 3e8:
        return None
    bwd = op == "qk_norm_bwd"
    D, R = case["headdim"], case["rotary"] // 2
    res = {}
    for n in ("q", "k"):
        x = s[n].double().contiguous().requires_grad_(bwd)
        w = s[n + "_w"].double().requires_grad_(bwd) if s[n + "_w"] is not None else None
        if case["norm"] == "rms":
            y = F.rms_norm(x, (D,), w, s["eps"])
        else:
            y = x / torch.sqrt(x.square().sum(-1, keepdim=True) + s["eps"])
            y = y * w if w is not None else y
        if R:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                               torch.outer(s["pos"].double(), s["freq"].double()))[:, None]
            pairs = y[..., :2 * R].unflatten(-1, (R, 2) if case["interleaved"] else (2, R))
            if not case["interleaved"]:
                pairs = pairs.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            if not case["interleaved"]:
                z = z.transpose(-1, -2)
            y = torch.cat([z.flatten(-2), y[..., 2 * R:]], -1)
        if not bwd:
            res[n] = y
            continue
        (y * s["d" + n].double()).sum().backward()
        res[n], res[n + "_weight"] = x.grad, w.grad if w is not None else None
    if not bwd:
        return res["q"], res["k"]
    return {k: res[k] for k in ("q", "k", "q_weight", "k_weight")}


def _exact_delta(case, s):
    """The recurrence, one token of every sequence at a time; sequences that have ended take
    steps that change nothing (beta 0, decay 1)."""
    b, T, lens = _lens(case)
    H, G, P, N, n = (*(case[k] for k in ("heads", "groups", "headdim", "dstate")), len(lens))
    longest = max(lens)
    # 40 passes over the states a token backward, 12 forward, at least 6 us each
    ops = 40 if case["op"] == "delta_bwd" else 12
    if longest * ops * max(6e-6, n * H * P * N * 8 / 3e12) > 15:
        return None
    dev = s["q"].device
    starts = [sum(lens[:i]) for i in range(n)]

    def rows(x, heads):
        """(longest, sequences, H, ...) in fp64, zeros behind a sequence's end."""
        x = x.flatten(0, 1)
        out = torch.zeros((longest, n) + tuple(x.shape[1:]), dtype=torch.float64, device=dev)
        for i, (at, m) in enumerate(zip(starts, lens)):
            out[:m, i] = x[at:at + m].double()
        return out if heads == H else out.repeat_interleave(H // heads, 2)

    def packed(x, like, heads):
        if heads != H:
            x = x.unflatten(2, (heads, H // heads)).sum(3)
        return torch.cat([x[:m, i] for i, m in enumerate(lens)]).reshape(like.shape)

    q, k, v = rows(s["q"], G), rows(s["k"], G), rows(s["v"], H)
    a, beta = torch.exp(rows(s["g"], H)), rows(s["beta"], H)
    S = s["init"].double() if s["init"] is not None else \
        torch.zeros((n, H, P, N), dtype=torch.float64, device=dev)

    def step(S, t):
        S = S * a[t][..., None, None]
        w = beta[t][..., None] * (v[t] - (S @ k[t][..., None])[..., 0])
        return S + w[..., None] * k[t][..., None, :]

    if case["op"] == "delta_fwd":
        out = torch.zeros((longest, n, H, P), dtype=torch.float64, device=dev)
        for t in range(longest):
            S = step(S, t)
            out[t] = s["scale"] * (S @ q[t][..., None])[..., 0]
        return packed(out, s["v"], H), S if case["final"] else None
    # states every `gap` tokens, then a segment's states again while its tokens are walked back
    gap = max(1, min(64, int(16e9 // (n * H * P * N * 8))))
    keep = []
    for t in range(longest):
        if t % gap == 0:
            keep.append(S.clone())
        S = step(S, t)
    do = rows(s["dout"], H)
    dS = s["dfinal"].double() if s["dfinal"] is not None else torch.zeros_like(S)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    da, db = torch.zeros_like(a), torch.zeros_like(beta)
    for at in reversed(range(0, longest, gap)):
        seg = [keep.pop()]
        for t in range(at, min(at + gap, longest)):
            seg.append(step(seg[-1], t))
        for t in reversed(range(at, min(at + gap, longest))):
            St, Sp = seg[t - at + 1], seg[t - at]
            kc, kr = k[t][..., None], k[t][..., None, :]
            dq[t] = s["scale"] * (St.transpose(-1, -2) @ do[t][..., None])[..., 0]
            dS = dS + s["scale"] * do[t][..., None] * q[t][..., None, :]
            read = (Sp @ kc)[..., 0]                         # S_(t-1) k
            miss = v[t] - a[t][..., None] * read
            dw = (dS @ kc)[..., 0]
            dk[t] = (dS.transpose(-1, -2) @ (beta[t][..., None] * miss)[..., None])[..., 0]
            db[t] = (dw * miss).sum(-1)
            dv[t] = beta[t][..., None] * dw
            # a S_(t-1) reaches the state directly and through what is read from it
            back = dS - dv[t][..., None] * kr
            dk[t] -= a[t][..., None] * (Sp.transpose(-1, -2) @ dv[t][..., None])[..., 0]
            da[t] = (back * Sp).sum((-1, -2))
            dS = a[t][..., None, None] * back
    return {"q": packed(dq, s["q"], G), "k": packed(dk, s["k"], G), "v": packed(dv, s["v"], H),
            "g": packed(da * a, s["g"], H), "beta": packed(db, s["beta"], H),
            "initial_states": dS if s["init"] is not None else None}
