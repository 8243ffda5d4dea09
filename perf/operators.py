"""What is measured of the operators around the scan in a Mamba layer.

The causal convolution, the selective scan with a decay per channel and state,
the gated norm after the scan and the residual norm before a block: each in its
forward, backward and (where it has one) single-token form.  ``run`` computes a
pass either in plain torch operations (``own`` false) or through the package's
entry points (``own`` true); ``exact`` is the same pass in 64 bits, written from
the definition over sequences padded side by side, its gradients by autograd.
"""
import math
import random

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def _conv(name, kind, dtype, batch, seqlen, channels, width=4, nseqs=0, state=False, silu=True, sliced=False):
    return {"name": name, "op": "conv", "pass": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen,
            "channels": channels, "width": width, "nseqs": nseqs, "state": state, "silu": silu, "sliced": sliced}


def _scan(name, kind, dtype, batch, seqlen, channels, dstate=16, groups=1, nseqs=0, state=False, gate=True,
          softplus=True, sliced=False):
    return {"name": name, "op": "scan", "pass": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen,
            "channels": channels, "dstate": dstate, "groups": groups, "nseqs": nseqs, "state": state,
            "gate": gate, "softplus": softplus, "sliced": sliced}


def _gated(name, kind, dtype, x_dtype, rows, channels, groups=1, gate_first=True, sliced=False):
    return {"name": name, "op": "gated", "pass": kind, "dtype": dtype, "x_dtype": x_dtype, "rows": rows,
            "channels": channels, "groups": groups, "gate_first": gate_first, "sliced": sliced}


def _residual(name, kind, dtype, rows, channels, residual=True, scale=False):
    return {"name": name, "op": "residual", "pass": kind, "dtype": dtype, "rows": rows, "channels": channels,
            "residual": residual, "scale": scale}


def listed():
    return [
        # prefill or training of the 2.7B layer: x, B and C of the scan (80 heads of 64 channels and twice 128
        # state columns) convolved as one slice of the input projection's output
        _conv("conv_prompt_bf16", "forward", "bf16", 4, 4096, 5376, sliced=True),
        # the same layer's training step on rows packed with eight sequences each, carried on from earlier pieces
        _conv("conv_backward_bf16", "backward", "bf16", 4, 4096, 5376, nseqs=8, state=True),
        # one decoded token for each of four requests of the 2.7B layer: latency
        _conv("conv_step_bf16", "step", "bf16", 4, 1, 5376),
        # prefill or training of a wide layer with a decay per channel and state
        _scan("scan_prompt_bf16", "forward", "bf16", 4, 4096, 5120, sliced=True),
        # one long document on a 130M-sized layer: few channels, so rows have to be split
        _scan("scan_long_bf16", "forward", "bf16", 1, 16384, 1536),
        # training of a 130M-sized layer
        _scan("scan_backward_bf16", "backward", "bf16", 8, 2048, 1536),
        # packed fp32 training of odd sizes with larger states, two groups and initial states
        _scan("scan_packed_backward_f32", "backward", "f32", 2, 777, 650, dstate=32, groups=2, nseqs=5, state=True),
        # one decoded token for each of 64 requests of the wide layer
        _scan("scan_step_bf16", "step", "bf16", 64, 1, 5120),
        # after the 2.7B layer's scan: its fp32 output gated by a slice of the projection, into the output projection
        _gated("gated_norm_bf16", "forward", "bf16", "f32", 16384, 5120, sliced=True),
        # training step of the same norm in eight groups
        _gated("gated_norm_backward_bf16", "backward", "bf16", "f32", 8192, 5120, groups=8),
        # before a block of the 2.7B layer (width 2560) in training: stream kept in fp32, learned branch scale
        _residual("residual_norm_backward_bf16", "backward", "bf16", 16384, 2560, scale=True),
        # before a block while four requests decode: latency
        _residual("residual_norm_decode_bf16", "forward", "bf16", 4, 2560),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng: random.Random):
    op = rng.choice(["conv", "conv", "scan", "scan", "scan", "gated", "residual"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "scan"):
        kind = rng.choice(["forward", "backward", "step"])
        batch = _spread(rng, 1, 64) if kind == "step" else _spread(rng, 1, 8)
        channels = _spread(rng, 32, 6144)
        if rng.random() < 0.5:
            channels = (channels + 31) // 32 * 32
        state = rng.random() < 0.5
    if op == "conv":
        # up to the listed training step's elements, 4 * 4096 * 5376 (fewer of the larger type)
        most = 88000000 if dtype == "bf16" else 60000000
        seqlen = 1 if kind == "step" else _spread(rng, 1, max(1, min(16384, most // (batch * channels))))
        nseqs = 0 if kind == "step" or rng.random() < 0.5 else _spread(rng, 1, min(32, seqlen))
        return _conv("", kind, dtype, batch, seqlen, channels, width=rng.choice([2, 3, 4]), nseqs=nseqs, state=state,
                     silu=rng.random() < 0.7, sliced=rng.random() < 0.4)
    if op == "scan":
        dstate = rng.choice([8, 16, 16, 32, 64])
        # up to the listed passes' state updates: 4 * 4096 * 5120 * 16 forward, 8 * 2048 * 1536 * 16 backward
        most = 1300000000 if kind == "forward" else 400000000
        longest = 16384 if kind == "forward" else 4096
        seqlen = 1 if kind == "step" else _spread(rng, 1, max(1, min(longest, most // (batch * channels * dstate))))
        nseqs = 0 if kind == "step" or rng.random() < 0.5 else _spread(rng, 1, min(32, seqlen))
        groups = rng.choice([g for g in (1, 1, 2, 3, 4) if channels % g == 0])
        return _scan("", kind, dtype, batch, seqlen, channels, dstate=dstate, groups=groups, nseqs=nseqs, state=state,
                     gate=rng.random() < 0.6, softplus=rng.random() < 0.7, sliced=rng.random() < 0.4)
    kind = rng.choice(["forward", "backward"])
    groups = rng.choice([1, 1, 2, 4, 8]) if op == "gated" else 1
    channels = groups * _spread(rng, 16, 8192 // groups)
    rows = _spread(rng, 1, 41000000 // channels) if op == "gated" else _spread(rng, 1, 20000000 // channels)
    if op == "gated":
        x_dtype = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
        return _gated("", kind, dtype, x_dtype, rows, channels, groups=groups, gate_first=rng.random() < 0.6,
                      sliced=rng.random() < 0.4)
    return _residual("", kind, dtype, rows, channels, residual=rng.random() < 0.8, scale=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs
def _slice(t, wanted):
    """The values of ``t`` as a slice of a wider projection's output, or as they are."""
    if not wanted:
        return t
    wide = torch.zeros(t.shape[:-1] + (t.shape[-1] + 128,), dtype=t.dtype, device=t.device)
    part = wide[..., 64:64 + t.shape[-1]]
    part.copy_(t)
    return part


def _ids(case, seed):
    """Sequence ids (batch, seqlen), or None: each row cut into nseqs pieces at random places."""
    if not case["nseqs"]:
        return None
    rng = random.Random(seed)
    T, k = case["seqlen"], case["nseqs"]
    rows = []
    for r in range(case["batch"]):
        cuts = [0] + sorted(rng.sample(range(1, T), k - 1)) + [T]
        for i in range(k):
            rows += [r * k + i] * (cuts[i + 1] - cuts[i])
    return torch.tensor(rows, dtype=torch.int32).view(case["batch"], T).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * std + mean

    def uniform(low, high, *shape):
        return torch.rand(shape, generator=gen, device="cuda") * (high - low) + low

    typ, D, kind = TYPES[case["dtype"]], case["channels"], case["pass"]
    s = dict(case)
    if case["op"] == "conv":
        b, T, K = case["batch"], case["seqlen"], case["width"]
        ids = _ids(case, seed)
        n = b * (case["nseqs"] or 1)
        s.update(x=_slice(normal(b, T, D).to(typ), case["sliced"]), weight=uniform(-K ** -0.5, K ** -0.5, D, K),
                 bias=normal(D, std=0.1), ids=ids, n=n, init=None)
        if case["state"] or kind == "step":
            s["init"] = normal(n, K - 1, D)
        if kind == "step":
            s["x"] = s["x"].view(b, D)
            s["next"] = torch.empty_like(s["init"])
        if kind == "backward":
            s.update(dy=normal(b, T, D), dfinal=normal(n, K - 1, D) if case["state"] else None)
    elif case["op"] == "scan":
        b, T, N, G = case["batch"], case["seqlen"], case["dstate"], case["groups"]
        ids = _ids(case, seed)
        n = b * (case["nseqs"] or 1)
        A_log = torch.arange(1, N + 1, device="cuda").float().log().expand(D, N) + normal(D, N, std=0.1)
        s.update(x=_slice(normal(b, T, D).to(typ), case["sliced"]), A_log=A_log.contiguous(), D=normal(D, std=0.1, mean=1.0),
                 B=_slice(normal(b, T, G * N, std=N ** -0.5).to(typ), case["sliced"]).unflatten(-1, (G, N)),
                 C=_slice(normal(b, T, G * N).to(typ), case["sliced"]).unflatten(-1, (G, N)),
                 z=_slice(normal(b, T, D).to(typ), case["sliced"]) if case["gate"] else None, ids=ids, n=n, init=None)
        if case["softplus"]:
            s.update(dt=uniform(-4.0, 1.0, b, T, D).to(typ), dt_bias=uniform(-1.0, 0.0, D))
        else:
            s.update(dt=torch.exp(uniform(math.log(1e-3), math.log(0.1), b, T, D)).to(typ), dt_bias=None)
        if case["state"] or kind == "step":
            s["init"] = normal(n, D, N, std=0.5)
        if kind == "step":
            for k in ("x", "dt", "z", "B", "C"):
                if s[k] is not None:
                    s[k] = s[k].squeeze(1)
            s["next"] = torch.empty_like(s["init"])
        if kind == "backward":
            s.update(dy=normal(b, T, D), dfinal=normal(n, D, N, std=0.5) if case["state"] else None)
    elif case["op"] == "gated":
        M = case["rows"]
        s.update(x=normal(M, D).to(TYPES[case["x_dtype"]]), z=_slice(normal(M, D).to(typ), case["sliced"]),
                 weight=normal(D, std=0.1, mean=1.0), dout=normal(M, D) if kind == "backward" else None)
    else:
        M = case["rows"]
        s.update(x=normal(M, D).to(typ), weight=normal(D, std=0.1, mean=1.0),
                 stream=normal(M, D, std=2.0) if case["residual"] or kind == "backward" else None,
                 gain=normal(D, std=0.1, mean=0.5) if case["scale"] else None)
        if kind == "backward":
            s.update(dout=normal(M, D), dstream=normal(M, D) if case["residual"] else None)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _calls(state)
    return _plain(state)


def _calls(s):
    import mamba_ssd_scan_chunked_amd as ssd
    kind = s["pass"]
    if s["op"] == "conv":
        if kind == "step":
            y = ssd.causal_conv_step(s["x"], s["weight"], s["bias"], s["init"], silu=s["silu"], state_out=s["next"])
            return {"y": y, "state": s["next"]}
        seqs = {"init_state": s["init"], "seq_idx": s["ids"], "nseqs": s["n"], "silu": s["silu"]}
        if kind == "forward":
            y, final = ssd.causal_conv(s["x"], s["weight"], s["bias"], **seqs)
            return {"y": y, "final": final}
        return ssd.causal_conv_backward(s["x"], s["weight"], s["dy"], s["bias"], dfinal=s["dfinal"], **seqs)
    if s["op"] == "scan":
        if kind == "step":
            y = ssd.selective_step(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["D"], s["init"], z=s["z"],
                                   dt_bias=s["dt_bias"], dt_softplus=s["softplus"], state_out=s["next"])
            return {"y": y, "state": s["next"]}
        more = {"D": s["D"], "z": s["z"], "init_state": s["init"], "seq_idx": s["ids"], "nseqs": s["n"],
                "dt_bias": s["dt_bias"], "dt_softplus": s["softplus"]}
        if kind == "forward":
            y, final = ssd.selective_scan(s["x"], s["dt"], s["A_log"], s["B"], s["C"], **more)
            return {"y": y, "final": final}
        return ssd.selective_scan_backward(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["dy"], dfinal=s["dfinal"],
                                           **more)
    if s["op"] == "gated":
        size = s["channels"] // s["groups"]
        if kind == "forward":
            return ssd.gated_norm(s["x"], s["z"], s["weight"], group_size=size, eps=EPS, gate_first=s["gate_first"])
        return ssd.gated_norm_backward(s["x"], s["z"], s["weight"], s["dout"], group_size=size, eps=EPS,
                                       gate_first=s["gate_first"])
    if kind == "forward":
        out, stream = ssd.residual_norm(s["x"], s["stream"], s["weight"], scale=s["gain"], eps=EPS)
        return {"out": out, "residual": stream}
    return ssd.residual_norm_backward(s["x"], s["stream"], s["weight"], s["dout"], dresidual_out=s["dstream"],
                                      scale=s["gain"], eps=EPS)


def _places(s):
    """Per token: its sequence id and its place in the sequence; per sequence: first token and length (flat tokens)."""
    b, T, n = s["batch"], s["seqlen"], s["n"]
    if s["ids"] is None:
        seq = torch.arange(b, device="cuda").repeat_interleave(T, output_size=b * T)
    else:
        seq = s["ids"].view(-1).long()
    length = torch.zeros(n, dtype=torch.long, device="cuda").scatter_add_(0, seq, torch.ones_like(seq))
    first = length.cumsum(0) - length
    return seq, torch.arange(b * T, device="cuda") - first[seq], first, length


def _silu(v):
    return v / (1 + torch.exp(-v))


def _silu_slope(v):
    p = 1 / (1 + torch.exp(-v))
    return p * (1 + v * (1 - p))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain(s):
    if s["op"] == "conv":
        return _plain_conv_step(s) if s["pass"] == "step" else _plain_conv(s)
    if s["op"] == "scan":
        return _plain_scan_step(s) if s["pass"] == "step" else _plain_scan(s)
    return _plain_gated(s) if s["op"] == "gated" else _plain_residual(s)


def _plain_conv_step(s):
    window = torch.cat([s["init"], s["x"].float()[:, None]], 1)
    pre = (window * s["weight"].t()).sum(1) + s["bias"]
    return {"y": (_silu(pre) if s["silu"] else pre).to(s["x"].dtype), "state": window[:, 1:].contiguous()}


def _plain_conv(s):
    b, T, D, K, n = s["batch"], s["seqlen"], s["channels"], s["width"], s["n"]
    x = s["x"].float().reshape(b * T, D)
    seq, place, first, length = _places(s)
    token = torch.arange(b * T, device="cuda")

    def lagged(j):
        # the input j tokens back: of the same sequence, else of its initial state, else zero
        inside = (place >= j)[:, None]
        before = 0.0 if s["init"] is None else s["init"][seq, (K - 1 + place - j).clamp(0, K - 2)]
        return torch.where(inside, x[(token - j).clamp(min=0)], before)

    pre = s["bias"] + sum(s["weight"][:, K - 1 - j] * (lagged(j) if j else x) for j in range(K))
    last = first + length - (K - 1)           # flat token of the final state's first row
    if s["pass"] == "forward":
        y = (_silu(pre) if s["silu"] else pre).to(s["x"].dtype).view(b, T, D)
        rows = []
        for i in range(K - 1):
            at = length - (K - 1) + i         # place in the sequence; negative: still the initial state's
            before = 0.0 if s["init"] is None else s["init"][torch.arange(n, device="cuda"), (K - 1 + at).clamp(0, K - 2)]
            rows.append(torch.where((at >= 0)[:, None], x[(last + i).clamp(min=0)], before))
        return {"y": y, "final": torch.stack(rows, 1)}
    g = s["dy"].view(b * T, D) * (_silu_slope(pre) if s["silu"] else 1.0)
    dx, dinit = torch.zeros_like(x), torch.zeros(n, K - 1, D, device="cuda")
    dweight = torch.empty_like(s["weight"])
    for j in range(K):
        dweight[:, K - 1 - j] = (g * (lagged(j) if j else x)).sum(0)
        part = g * s["weight"][:, K - 1 - j]
        inside = (place >= j)[:, None]
        dx.index_add_(0, (token - j).clamp(min=0), torch.where(inside, part, 0.0))
        for p in range(j):                    # token p of each sequence reaches j back, into the initial state
            hit = (length > p)[:, None]
            dinit[:, K - 1 + p - j] += torch.where(hit, part[(first + p).clamp(max=b * T - 1)], 0.0)
    if s["dfinal"] is not None:
        which = torch.arange(n, device="cuda")
        for i in range(K - 1):
            at = length - (K - 1) + i
            inside = (at >= 0)[:, None]
            dx.index_add_(0, (last + i).clamp(min=0), torch.where(inside, s["dfinal"][:, i], 0.0))
            dinit.index_put_((which, (K - 1 + at).clamp(0, K - 2)), torch.where(inside, 0.0, s["dfinal"][:, i]),
                             accumulate=True)
    return {"dx": dx.view(b, T, D), "dweight": dweight, "dbias": g.sum(0), "dinit": dinit}


def _plain_scan_step(s):
    D, G = s["channels"], s["groups"]
    step = s["dt"].float() + (0.0 if s["dt_bias"] is None else s["dt_bias"])
    step = _softplus(step) if s["softplus"] else step
    x = s["x"].float()
    B, C = (s[k].float().repeat_interleave(D // G, 1) for k in ("B", "C"))
    h = torch.exp(step[..., None] * -torch.exp(s["A_log"])) * s["init"] + (step * x)[..., None] * B
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(s["x"].dtype), "state": h}


def _plain_scan(s):
    b, T, D, N, G, n = s["batch"], s["seqlen"], s["channels"], s["dstate"], s["groups"], s["n"]
    raw = s["dt"].float() + (0.0 if s["dt_bias"] is None else s["dt_bias"])
    step = _softplus(raw) if s["softplus"] else raw
    x, A = s["x"].float(), -torch.exp(s["A_log"])
    u = step * x
    B, C = s["B"].float(), s["C"].float()
    seq, place, _, _ = _places(s)
    seq, starts = seq.view(b, T), (place == 0).view(b, T, 1, 1)
    init = torch.zeros(n, D, N, device="cuda") if s["init"] is None else s["init"]
    wide = (b, G, D // G, N)                  # channels by group

    def over(t, v):                           # B_t or C_t, for each channel of its group
        return v[:, t, :, None, :].expand(wide).reshape(b, D, N)

    h, final, y = init[seq[:, 0]], init.clone(), torch.empty(b, T, D, device="cuda")
    back = s["pass"] == "backward"
    before = torch.empty(T, b, D, N, device="cuda") if back else None
    after = torch.empty(T, b, D, N, device="cuda") if back else None
    for t in range(T):
        if s["ids"] is not None:
            h = torch.where(starts[:, t], init[seq[:, t]], h)
        if back:
            before[t] = h
        h = torch.exp(step[:, t, :, None] * A) * h + u[:, t, :, None] * over(t, B)
        if back:
            after[t] = h
        if s["ids"] is not None:
            final[seq[:, t]] = h
        y[:, t] = (h * over(t, C)).sum(-1)
    if s["ids"] is None:
        final = h
    y += s["D"] * x
    if not back:
        if s["z"] is not None:
            y = y * _silu(s["z"].float())
        return {"y": y.to(s["x"].dtype), "final": final}

    out = {}
    dy = s["dy"]
    if s["z"] is not None:
        z = s["z"].float()
        out["dz"] = dy * y * _silu_slope(z)
        dy = dy * _silu(z)
    dfinal = torch.zeros(n, D, N, device="cuda") if s["dfinal"] is None else s["dfinal"]
    ends = torch.ones(b, T, 1, 1, dtype=torch.bool, device="cuda")
    ends[:, :-1] = starts[:, 1:]
    dstep, du = torch.empty(b, T, D, device="cuda"), torch.empty(b, T, D, device="cuda")
    dB, dC = torch.empty(b, T, G, N, device="cuda"), torch.empty(b, T, G, N, device="cuda")
    dA, dinit = torch.zeros(b, D, N, device="cuda"), torch.zeros(n, D, N, device="cuda")
    q = torch.zeros(b, D, N, device="cuda")   # gradient reaching the state after token t from later tokens
    for t in range(T - 1, -1, -1):
        if s["ids"] is not None or t == T - 1:
            q = torch.where(ends[:, t], dfinal[seq[:, t]], q)
        q = q + dy[:, t, :, None] * over(t, C)
        dC[:, t] = (dy[:, t, :, None] * after[t]).view(wide).sum(2)
        dB[:, t] = (q * u[:, t, :, None]).view(wide).sum(2)
        du[:, t] = (q * over(t, B)).sum(-1)
        q = q * torch.exp(step[:, t, :, None] * A)
        m = q * before[t]
        dstep[:, t] = (m * A).sum(-1)
        dA += m * step[:, t, :, None]
        if s["ids"] is not None or t == 0:    # the last write for a sequence is the one at its first token
            dinit[seq[:, t]] = q
    dstep += du * x
    draw_ = dstep / (1 + torch.exp(-raw)) if s["softplus"] else dstep
    out.update(dx=du * step + s["D"] * dy, ddt=draw_, dA_log=dA.sum(0) * A, dB=dB, dC=dC, dD=(dy * x).sum((0, 1)),
               dinit=dinit, ddt_bias=draw_.sum((0, 1)))
    return out


def _plain_gated(s):
    M, D, G = s["rows"], s["channels"], s["groups"]
    x, z, w = s["x"].float(), s["z"].float(), s["weight"]

    def mean(v):
        return v.view(M, G, D // G).mean(-1, keepdim=True).expand(M, G, D // G).reshape(M, D)

    gate = _silu(z)
    u = x * gate if s["gate_first"] else x
    r = torch.rsqrt(mean(u * u) + EPS)
    if s["pass"] == "forward":
        out = u * r * w
        return (out if s["gate_first"] else out * gate).to(s["z"].dtype)
    e = s["dout"] if s["gate_first"] else s["dout"] * gate
    hat = u * r
    du = r * (e * w - hat * mean(e * w * hat))
    if s["gate_first"]:
        return {"dx": du * gate, "dz": du * x * _silu_slope(z), "dweight": (e * hat).sum(0)}
    return {"dx": du, "dz": s["dout"] * hat * w * _silu_slope(z), "dweight": (e * hat).sum(0)}


def _plain_residual(s):
    x, w = s["x"].float(), s["weight"]
    if s["pass"] == "forward":
        stream = x if s["gain"] is None else x * s["gain"]
        if s["stream"] is not None:
            stream = s["stream"] + stream
        r = torch.rsqrt((stream * stream).mean(-1, keepdim=True) + EPS)
        return {"out": (stream * r * w).to(s["x"].dtype), "residual": stream}
    stream, e = s["stream"], s["dout"]
    r = torch.rsqrt((stream * stream).mean(-1, keepdim=True) + EPS)
    hat = stream * r
    d = r * (e * w - hat * (e * w * hat).mean(-1, keepdim=True))
    if s["dstream"] is not None:
        d = d + s["dstream"]
    out = {"dx": d if s["gain"] is None else d * s["gain"], "dresidual": d, "dweight": (e * hat).sum(0)}
    if s["gain"] is not None:
        out["dscale"] = (d * x).sum(0)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e, D, kind = (2 if case["dtype"] == "bf16" else 4), case["channels"], case["pass"]
    if case["op"] in ("conv", "scan"):
        m = case["batch"] * case["seqlen"]
        n = case["batch"] * (case["nseqs"] or 1)
        ids = 4 * m if case["nseqs"] else 0
        given = 1 if case["state"] or kind == "step" else 0
    if case["op"] == "conv":
        K = case["width"]
        state, params = 4 * n * (K - 1) * D, 4 * D * (K + 1)
        act = 5 if case["silu"] else 0
        if kind != "backward":
            return {"bytes": 2 * e * m * D + params + (1 + given) * state + ids, "flops": m * D * (2 * K + act)}
        return {"bytes": (e + 8) * m * D + 2 * params + (1 + 2 * given) * state + ids,
                "flops": m * D * (6 * K + 2 * act)}
    if case["op"] == "scan":
        N, G, gate = case["dstate"], case["groups"], 1 if case["gate"] else 0
        state, params = 4 * n * D * N, 4 * D * (N + 1 + (1 if case["softplus"] else 0))
        if kind != "backward":
            moved = e * m * ((3 + gate) * D + 2 * G * N)
            return {"bytes": moved + params + (1 + given) * state + ids, "flops": m * D * (7 * N + 10)}
        moved = m * ((e * (2 + gate) + 4 * (3 + gate)) * D + (2 * e + 8) * G * N)
        # the gradients include one for dt_bias, given or not
        return {"bytes": moved + params + 4 * D * (N + 2) + (1 + 2 * given) * state + ids,
                "flops": m * D * (20 * N + 30)}
    M = case["rows"]
    if case["op"] == "gated":
        ex = 2 if case["x_dtype"] == "bf16" else 4
        if kind == "forward":
            return {"bytes": M * D * (ex + 2 * e) + 4 * D, "flops": 10 * M * D}
        return {"bytes": M * D * (ex + e + 12) + 8 * D, "flops": 25 * M * D}
    res, gain = 1 if case["residual"] else 0, 1 if case["scale"] else 0
    if kind == "forward":
        return {"bytes": M * D * (2 * e + 4 + 4 * res) + 4 * D * (1 + gain), "flops": 6 * M * D}
    # x is read for the scale's gradient only; without a scale dx is dresidual
    return {"bytes": M * D * (8 + 4 * res + 4 + gain * (e + 4)) + 8 * D * (1 + gain), "flops": 15 * M * D}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    w = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    with torch.enable_grad():
        return {"conv": _exact_conv, "scan": _exact_scan, "gated": _exact_gated, "residual": _exact_residual}[
            case["op"]](w)


def _leaf(t):
    return t.detach().clone().requires_grad_()


def _padded(s):
    """Sequences side by side: for each, the flat token at every place and which places exist (n, longest)."""
    b, T = s["batch"], s["seqlen"]
    ids = [[r] * T for r in range(b)] if s["ids"] is None else s["ids"].tolist()
    where = [[] for _ in range(s["n"])]
    for r, row in enumerate(ids):
        for t, q in enumerate(row):
            where[q].append(r * T + t)
    longest = max(len(p) for p in where)
    index = torch.tensor([p + [0] * (longest - len(p)) for p in where], device="cuda")
    real = torch.tensor([[1] * len(p) + [0] * (longest - len(p)) for p in where], device="cuda").bool()
    return index, real


def _flat(s, index, real, padded):
    """Back from padded sequences to (batch, seqlen, ...)."""
    out = padded.new_zeros((s["batch"] * s["seqlen"],) + padded.shape[2:])
    out = out.index_put((index[real],), padded[real])
    return out.view((s["batch"], s["seqlen"]) + padded.shape[2:])


def _exact_conv(s):
    D, K, n = s["channels"], s["width"], s["n"]
    if s["pass"] == "step":
        s["x"], s["seqlen"], s["ids"] = s["x"][:, None], 1, None
    x, weight, bias = _leaf(s["x"]), _leaf(s["weight"]), _leaf(s["bias"])
    init = _leaf(torch.zeros(n, K - 1, D, dtype=torch.double, device="cuda") if s["init"] is None else s["init"])
    index, real = _padded(s)
    line = torch.cat([init, x.reshape(-1, D)[index]], 1)
    reach = index.shape[1]
    pre = bias
    for k in range(K):
        pre = pre + line[:, k:k + reach] * weight[:, k]
    y = _flat(s, index, real, pre * torch.sigmoid(pre) if s["silu"] else pre)
    tail = real.sum(1)[:, None] + torch.arange(K - 1, device="cuda")
    final = line[torch.arange(n, device="cuda")[:, None], tail]
    if s["pass"] == "step":
        return {"y": y.detach()[:, 0], "state": final.detach()}
    if s["pass"] == "forward":
        return {"y": y.detach(), "final": final.detach()}
    loss = (y * s["dy"]).sum() + (0.0 if s["dfinal"] is None else (final * s["dfinal"]).sum())
    return dict(zip(("dx", "dweight", "dbias", "dinit"), torch.autograd.grad(loss, (x, weight, bias, init))))


def _exact_scan(s):
    D, N, G, n = s["channels"], s["dstate"], s["groups"], s["n"]
    kind = s["pass"]
    if kind == "step":
        for k in ("x", "dt", "B", "C", "z"):
            s[k] = s[k] if s[k] is None else s[k][:, None]
        s["seqlen"], s["ids"] = 1, None
    grads = kind == "backward"
    leaf = _leaf if grads else (lambda t: t)
    x, dt, A_log, B, C = (leaf(s[k]) for k in ("x", "dt", "A_log", "B", "C"))
    skip, z = leaf(s["D"]), None if s["z"] is None else leaf(s["z"])
    zeros = torch.zeros(n, D, N, dtype=torch.double, device="cuda")
    init = leaf(zeros if s["init"] is None else s["init"])
    bias = leaf(torch.zeros(D, dtype=torch.double, device="cuda") if s["dt_bias"] is None else s["dt_bias"])
    step = dt + bias
    if s["softplus"]:
        step = torch.logaddexp(step, torch.zeros_like(step))
    index, real = _padded(s)
    A = -torch.exp(A_log)
    # a place beyond a sequence's end has step size zero: it leaves the state as it is
    step_p = step.reshape(-1, D)[index] * real[..., None]
    in_p = step_p * x.reshape(-1, D)[index]
    B_p, C_p = B.reshape(-1, G, N)[index], C.reshape(-1, G, N)[index]
    state, read = init.view(n, G, D // G, N), []
    A = A.view(G, D // G, N)
    for step_t, in_t, B_t, C_t in zip(step_p.unbind(1), in_p.unbind(1), B_p.unbind(1), C_p.unbind(1)):
        keep = torch.exp(step_t.view(n, G, -1, 1) * A)
        state = state * keep + in_t.view(n, G, -1, 1) * B_t[:, :, None]
        read.append(torch.matmul(state, C_t[..., None]).reshape(n, D))
    y = _flat(s, index, real, torch.stack(read, 1)) + skip * x
    if z is not None:
        y = y * z * torch.sigmoid(z)
    final = state.reshape(n, D, N)
    if kind == "step":
        return {"y": y[:, 0], "state": final}
    if kind == "forward":
        return {"y": y, "final": final}
    loss = (y * s["dy"]).sum() + (0.0 if s["dfinal"] is None else (final * s["dfinal"]).sum())
    names = ["dx", "ddt", "dA_log", "dB", "dC", "dD", "dinit", "ddt_bias"]
    leaves = [x, dt, A_log, B, C, skip, init, bias]
    if z is not None:
        names, leaves = ["dz"] + names, [z] + leaves
    return dict(zip(names, torch.autograd.grad(loss, leaves)))


def _exact_gated(s):
    D, G = s["channels"], s["groups"]
    x, z, weight = _leaf(s["x"]), _leaf(s["z"]), _leaf(s["weight"])
    gate = z * torch.sigmoid(z)
    u = (x * gate if s["gate_first"] else x).unflatten(-1, (G, D // G))
    normed = (u / torch.sqrt((u ** 2).mean(-1, keepdim=True) + EPS)).flatten(-2) * weight
    out = normed if s["gate_first"] else normed * gate
    if s["pass"] == "forward":
        return out.detach()
    return dict(zip(("dx", "dz", "dweight"), torch.autograd.grad((out * s["dout"]).sum(), (x, z, weight))))


def _exact_residual(s):
    x, weight = _leaf(s["x"]), _leaf(s["weight"])
    if s["pass"] == "forward":
        stream = x * (1.0 if s["gain"] is None else s["gain"]) + (0.0 if s["stream"] is None else s["stream"])
        out = stream / torch.sqrt((stream ** 2).mean(-1, keepdim=True) + EPS) * weight
        return {"out": out.detach(), "residual": stream.detach()}
    stream = _leaf(s["stream"])
    out = stream / torch.sqrt((stream ** 2).mean(-1, keepdim=True) + EPS) * weight
    loss = (out * s["dout"]).sum() + (0.0 if s["dstream"] is None else (stream * s["dstream"]).sum())
    dstream, dweight = torch.autograd.grad(loss, (stream, weight))
    if s["gain"] is None:
        return {"dx": dstream, "dresidual": dstream, "dweight": dweight}
    return {"dx": dstream * s["gain"], "dresidual": dstream, "dweight": dweight, "dscale": (dstream * s["x"]).sum(0)}
