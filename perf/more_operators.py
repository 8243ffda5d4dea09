"""What is measured of the gated linear recurrence and of the norm with rotation.

The gated linear recurrence (one state per channel, its decay and its input scale
from gates of the same token) and the root-mean-square norm of the scan's keys and
queries, B and C, per head with the rotation by position: each in its forward and
backward form, the recurrence for single tokens too.  ``run`` computes a pass either
in plain torch operations (``own`` false) or through the package's entry points
(``own`` true); ``exact`` is the same pass in 64 bits, written from the definition:
the recurrence token by token over sequences padded side by side, the rotation as a
product of complex numbers, gradients by autograd.
"""
import math
import random

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def _recurrence(name, kind, dtype, batch, seqlen, channels, nseqs=0, state=False, gate=False, sliced=False):
    return {"name": name, "op": "recurrence", "pass": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen,
            "channels": channels, "nseqs": nseqs, "state": state, "gate": gate, "sliced": sliced}


def _rotary(name, kind, dtype, batch, seqlen, b_heads, c_heads, headdim, rotary, interleaved=False, start=0,
            nseqs=0, sliced=False):
    return {"name": name, "op": "rotary", "pass": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen,
            "b_heads": b_heads, "c_heads": c_heads, "headdim": headdim, "rotary": rotary, "interleaved": interleaved,
            "start": start, "nseqs": nseqs, "sliced": sliced}


def listed():
    return [
        # prefill or training of a layer as wide as the 2.7B model: gates and input are slices of one projection
        _recurrence("recurrence_prompt_bf16", "forward", "bf16", 4, 4096, 2560, sliced=True),
        # one long document on a 130M-sized layer with an output gate: few channels, so the row has to be split
        _recurrence("recurrence_long_bf16", "forward", "bf16", 1, 16384, 1536, gate=True),
        # training step of the wide layer on rows packed with eight sequences each, carried on from earlier pieces
        _recurrence("recurrence_backward_bf16", "backward", "bf16", 4, 4096, 2560, nseqs=8, state=True),
        # training of a 130M-sized layer with an output gate
        _recurrence("recurrence_gate_backward_bf16", "backward", "bf16", 8, 2048, 1536, gate=True),
        # packed fp32 training of odd sizes
        _recurrence("recurrence_packed_backward_f32", "backward", "f32", 2, 777, 650, nseqs=5, state=True),
        # one decoded token for each of 64 requests of the wide layer: latency
        _recurrence("recurrence_step_bf16", "step", "bf16", 64, 1, 2560, gate=True),
        # prefill or training of the 2.7B layer: one group of 128 state columns for B and for C, slices of the
        # convolution's output, whole heads rotated
        _rotary("rotary_prompt_bf16", "forward", "bf16", 4, 4096, 1, 1, 128, 128, sliced=True),
        # a prompt with 32 query heads on 8 shared key heads, from a far position on, pairs side by side
        _rotary("rotary_heads_bf16", "forward", "bf16", 2, 4096, 8, 32, 128, 128, interleaved=True, start=1000000),
        # training step with eight groups of 128 state columns, packed sequences: positions start again
        _rotary("rotary_backward_bf16", "backward", "bf16", 4, 4096, 8, 8, 128, 128, nseqs=8),
        # fp32 training of odd sizes, half of each head rotated
        _rotary("rotary_part_backward_f32", "backward", "f32", 3, 777, 3, 6, 80, 40),
        # one decoded token for each of four requests of the 2.7B layer, at their own positions: latency
        _rotary("rotary_decode_bf16", "forward", "bf16", 4, 1, 1, 1, 128, 128, start=5000),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng: random.Random):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.55:
        kind = rng.choice(["forward", "backward", "step"])
        batch = _spread(rng, 1, 256) if kind == "step" else _spread(rng, 1, 8)
        channels = _spread(rng, 32, 5120)
        if rng.random() < 0.5:
            channels = (channels + 31) // 32 * 32
        # up to the listed passes' elements, 4 * 4096 * 2560 (fewer of the larger type)
        most = 40000000 if dtype == "bf16" else 24000000
        seqlen = 1 if kind == "step" else _spread(rng, 1, max(1, min(16384, most // (batch * channels))))
        nseqs = 0 if kind == "step" or rng.random() < 0.5 else _spread(rng, 1, min(32, seqlen))
        return _recurrence("", kind, dtype, batch, seqlen, channels, nseqs=nseqs, state=rng.random() < 0.5,
                           gate=rng.random() < 0.5, sliced=rng.random() < 0.4)
    kind = rng.choice(["forward", "backward"])
    b_heads = rng.choice([1, 1, 2, 3, 4, 8])
    c_heads = b_heads * rng.choice([1, 1, 2, 4])
    headdim = rng.choice([16, 32, 64, 64, 72, 80, 96, 100, 128, 128, 192, 256])
    rotary = rng.choice([headdim, headdim, headdim // 2 // 2 * 2])
    # up to the listed passes' elements, 8192 tokens of 40 heads of 128 forward, 16384 of 16 backward
    most = (40000000 if kind == "forward" else 32000000) // (1 if dtype == "bf16" else 2)
    tokens = _spread(rng, 1, min(32768, most // ((b_heads + c_heads) * headdim)))
    batch = rng.choice([n for n in (1, 2, 3, 4) if n <= tokens])
    seqlen = tokens // batch
    nseqs = 0 if rng.random() < 0.5 else _spread(rng, 1, min(32, seqlen))
    return _rotary("", kind, dtype, batch, seqlen, b_heads, c_heads, headdim, rotary,
                   interleaved=rng.random() < 0.4, start=rng.choice([0, 0, _spread(rng, 1, 4000000)]),
                   nseqs=nseqs, sliced=rng.random() < 0.4)


# ------------------------------------------------------------------ the inputs
def _slice(t, wanted):
    """The values of ``t`` as a slice of a wider projection's output, or as they are."""
    if not wanted:
        return t
    wide = torch.zeros(t.shape[:-1] + (t.shape[-1] + 128,), dtype=t.dtype, device=t.device)
    part = wide[..., 64:64 + t.shape[-1]]
    part.copy_(t)
    return part


def _lengths(case, seed):
    """Tokens of each sequence, row by row: each row cut into nseqs pieces at random places."""
    rng = random.Random(seed)
    T, k = case["seqlen"], case["nseqs"] or 1
    rows = []
    for _ in range(case["batch"]):
        cuts = [0] + sorted(rng.sample(range(1, T), k - 1)) + [T]
        rows.append([cuts[i + 1] - cuts[i] for i in range(k)])
    return rows


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * std + mean

    typ, kind, b, T = TYPES[case["dtype"]], case["pass"], case["batch"], case["seqlen"]
    rows = _lengths(case, seed)
    flat = torch.tensor([n for row in rows for n in row])
    s = dict(case)
    if case["op"] == "recurrence":
        D, n = case["channels"], flat.numel()
        ids = torch.arange(n, dtype=torch.int32).repeat_interleave(flat).view(b, T).cuda() if case["nseqs"] else None
        # decays of a whole gate spread from 0.9 to 0.999 to the eighth power, as such layers start from
        rate = -8 * torch.log(torch.rand(D, generator=gen, device="cuda") * 0.099 + 0.9)
        s.update(A_log=rate.log(), ids=ids, n=n, init=normal(n, D) if case["state"] or kind == "step" else None)
        for name in ("x", "r", "i") + (("z",) if case["gate"] else ()):
            s[name] = _slice(normal(b, T, D).to(typ), case["sliced"])
        s.setdefault("z", None)
        if kind == "step":
            for k in ("x", "r", "i", "z"):
                s[k] = s[k] if s[k] is None else s[k].squeeze(1)
            s["next"] = torch.empty_like(s["init"])
        if kind == "backward":
            s.update(dy=normal(b, T, D), dfinal=normal(n, D) if case["state"] else None)
        return s
    N, half = case["headdim"], case["rotary"] // 2
    s["freqs"] = (10000.0 ** (-torch.arange(half, dtype=torch.double) / half)).float().cuda()
    s["positions"] = None
    if case["nseqs"] or case["start"] or T == 1:
        place = torch.cat([torch.arange(n) for row in rows for n in row]).view(b, T)
        # every row from a position of its own
        first = torch.tensor([random.Random(seed + r).randrange(case["start"] + 1) for r in range(b)])
        s["positions"] = (place + case["start"] + first[:, None]).int().cuda()
    for k, heads in (("B", case["b_heads"]), ("C", case["c_heads"])):
        s[k] = _slice(normal(b, T, heads * N, std=1.5).to(typ), case["sliced"]).unflatten(-1, (heads, N))
        s[k.lower() + "_weight"] = normal(N, std=0.1, mean=1.0)
        if kind == "backward":
            s["d" + k] = normal(b, T, heads, N)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _calls(state)
    return _plain(state)


def _calls(s):
    import mamba_ssd_scan_chunked_amd as ssd
    kind = s["pass"]
    if s["op"] == "recurrence":
        if kind == "step":
            y = ssd.gated_recurrence_step(s["x"], s["r"], s["i"], s["A_log"], s["init"], z=s["z"], state_out=s["next"])
            return {"y": y, "state": s["next"]}
        more = {"z": s["z"], "init_state": s["init"], "seq_idx": s["ids"], "nseqs": s["n"]}
        if kind == "forward":
            y, final = ssd.gated_recurrence(s["x"], s["r"], s["i"], s["A_log"], **more)
            return {"y": y, "final": final}
        return ssd.gated_recurrence_backward(s["x"], s["r"], s["i"], s["A_log"], s["dy"], dfinal=s["dfinal"], **more)
    more = {"positions": s["positions"], "interleaved": s["interleaved"], "eps": EPS}
    args = (s["B"], s["C"], s["b_weight"], s["c_weight"], s["freqs"])
    if kind == "forward":
        B, C = ssd.rotary_norm(*args, **more)
        return {"B": B, "C": C}
    return ssd.rotary_norm_backward(*args, s["dB"], s["dC"], **more)


def _plain(s):
    if s["op"] == "rotary":
        return _plain_rotary(s)
    return _plain_step(s) if s["pass"] == "step" else _plain_recurrence(s)


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _gates(s):
    """Per token and channel: log of the decay, decay, scale of the input and gated input."""
    L = -torch.exp(s["A_log"]) * _sigmoid(s["r"].float())
    return L, torch.exp(L), torch.sqrt(-torch.expm1(2 * L)), _sigmoid(s["i"].float()) * s["x"].float()


def _plain_step(s):
    _, a, scale, u = _gates(s)
    h = a * s["init"] + scale * u
    y = h if s["z"] is None else h * s["z"].float() * _sigmoid(s["z"].float())
    return {"y": y.to(s["x"].dtype), "state": h}


def _running(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from zero, by doubling the reach."""
    reach, T = 1, a.shape[1]
    while reach < T:
        b = torch.cat([b[:, :reach], b[:, reach:] + a[:, reach:] * b[:, :-reach]], 1)
        a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return b


def _plain_recurrence(s):
    b, T, D, n = s["batch"], s["seqlen"], s["channels"], s["n"]
    L, a, scale, u = _gates(s)
    seq = torch.arange(n, device="cuda")[:, None].expand(b, T) if s["ids"] is None else s["ids"].long()
    fresh = torch.ones(b, T, dtype=torch.bool, device="cuda")
    fresh[:, 1:] = seq[:, 1:] != seq[:, :-1]
    last = torch.ones_like(fresh)
    last[:, :-1] = fresh[:, 1:]
    init = torch.zeros(n, D, device="cuda") if s["init"] is None else s["init"]
    added = scale * u
    added[fresh] += a[fresh] * init            # sequences begin in the order of their ids
    kept = torch.where(fresh[..., None], 0.0, a)
    h = _running(kept, added)
    gate = None if s["z"] is None else _sigmoid(s["z"].float())
    if s["pass"] == "forward":
        y = h if gate is None else h * s["z"].float() * gate
        return {"y": y.to(s["x"].dtype), "final": h[last]}
    out, g = {}, s["dy"]
    if gate is not None:
        z = s["z"].float()
        out["dz"] = g * h * gate * (1 + z * (1 - gate))
        g = g * z * gate
    if s["dfinal"] is not None:
        g = g.clone()
        g[last] += s["dfinal"]
    back = torch.cat([kept[:, 1:], torch.zeros(b, 1, D, device="cuda")], 1)
    g = _running(back.flip(1), g.flip(1)).flip(1)
    before = torch.cat([torch.zeros(b, 1, D, device="cuda"), h[:, :-1]], 1)
    before[fresh] = init
    i = _sigmoid(s["i"].float())
    ratio = torch.where(scale > 0, L / scale, 0.0)
    m = g * (L * a * before - u * a * a * ratio)
    out.update(dx=g * scale * i, dr=m / (1 + torch.exp(s["r"].float())), di=g * scale * u * (1 - i),
               dA_log=m.sum((0, 1)), dinit=(a * g)[fresh])
    return out


def _turns(s):
    """Cosine and sine (tokens, 1, rotary / 2) of every token's angles."""
    b, T = s["batch"], s["seqlen"]
    place = torch.arange(T, device="cuda").expand(b, T) if s["positions"] is None else s["positions"]
    angle = place.reshape(-1, 1, 1).double() * s["freqs"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _pairs(s, v):
    """(first members, second members, rest) of the last dimension."""
    R = s["rotary"]
    if s["interleaved"]:
        return v[..., 0:R:2], v[..., 1:R:2], v[..., R:]
    return v[..., :R // 2], v[..., R // 2:R], v[..., R:]


def _joined(s, p, q, rest):
    if s["interleaved"]:
        return torch.cat([torch.stack([p, q], -1).flatten(-2), rest], -1)
    return torch.cat([p, q, rest], -1)


def _plain_rotary(s):
    cos, sin = _turns(s)
    N = s["headdim"]
    out = {}
    for k in ("B", "C"):
        x, w = s[k].float().reshape(-1, s[k].shape[-2], N), s[k.lower() + "_weight"]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if s["pass"] == "forward":
            p, q, rest = _pairs(s, x * r * w)
            out[k] = _joined(s, p * cos - q * sin, p * sin + q * cos, rest).to(s[k].dtype).view(s[k].shape)
            continue
        p, q, rest = _pairs(s, s["d" + k].view(x.shape))
        e = _joined(s, p * cos + q * sin, q * cos - p * sin, rest)
        hat = x * r
        out["d" + k] = (r * (e * w - hat * (e * w * hat).mean(-1, keepdim=True))).view(s[k].shape)
        out["d" + k.lower() + "_weight"] = (e * hat).sum((0, 1))
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e, kind, m = (2 if case["dtype"] == "bf16" else 4), case["pass"], case["batch"] * case["seqlen"]
    if case["op"] == "recurrence":
        D, gate = case["channels"], 1 if case["gate"] else 0
        state = 4 * case["batch"] * (case["nseqs"] or 1) * D
        given = 1 if case["state"] or kind == "step" else 0
        other = (1 + given) * state + 4 * D + (4 * m if case["nseqs"] else 0)
        if kind != "backward":
            return {"bytes": m * D * e * (4 + gate) + other, "flops": m * D * (20 + 5 * gate)}
        # dinit is written, given or not
        return {"bytes": m * D * (e * (3 + gate) + 4 + 12 + 4 * gate) + other + given * state + 4 * D,
                "flops": m * D * (45 + 12 * gate)}
    values = m * (case["b_heads"] + case["c_heads"]) * case["headdim"]
    other = 8 * case["headdim"] + 2 * case["rotary"] + (4 * m if case["nseqs"] or case["start"] or case["seqlen"] == 1 else 0)
    if kind == "forward":
        return {"bytes": 2 * e * values + other, "flops": 7 * values}
    return {"bytes": (e + 8) * values + other + 8 * case["headdim"], "flops": 14 * values}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    w = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    with torch.enable_grad():
        return _exact_recurrence(w) if case["op"] == "recurrence" else _exact_rotary(w)


def _leaf(t):
    return t.detach().clone().requires_grad_()


def _exact_recurrence(s):
    D, n, kind = s["channels"], s["n"], s["pass"]
    if kind == "step":
        for k in ("x", "r", "i", "z"):
            s[k] = s[k] if s[k] is None else s[k][:, None]
    b, T = s["x"].shape[:2]
    leaf = _leaf if kind == "backward" else (lambda t: t)
    x, r, i, A_log = (leaf(s[k]) for k in ("x", "r", "i", "A_log"))
    z = None if s["z"] is None else leaf(s["z"])
    init = leaf(torch.zeros(n, D, dtype=torch.double, device="cuda") if s["init"] is None else s["init"])
    decay = torch.exp(-torch.exp(A_log) * torch.sigmoid(r))
    taken = torch.sqrt((1 - decay) * (1 + decay)) * torch.sigmoid(i) * x
    # sequences side by side, (longest, n): the flat token of every place, and which places exist
    where = [list(range(k * T, k * T + T)) for k in range(b)]
    if s["ids"] is not None:
        where = [[] for _ in range(n)]
        for token, k in enumerate(s["ids"].view(-1).tolist()):
            where[k].append(token)
    longest = max(len(p) for p in where)
    index = torch.tensor([p + [-1] * (longest - len(p)) for p in where], device="cuda").t()
    real = index >= 0
    decay_p = torch.where(real[..., None], decay.reshape(-1, D)[index.clamp(min=0)], 1.0)
    taken_p = torch.where(real[..., None], taken.reshape(-1, D)[index.clamp(min=0)], 0.0)
    state, states = init, []
    for decay_t, taken_t in zip(decay_p.unbind(0), taken_p.unbind(0)):
        state = decay_t * state + taken_t
        states.append(state)
    places = torch.stack(states)
    h = places.new_zeros(b * T, D).index_put((index[real],), places[real]).view(b, T, D)
    y = h if z is None else h * z * torch.sigmoid(z)
    if kind == "step":
        return {"y": y[:, 0], "state": state}
    if kind == "forward":
        return {"y": y, "final": state}
    loss = (y * s["dy"]).sum() + (0.0 if s["dfinal"] is None else (state * s["dfinal"]).sum())
    names, leaves = ["dx", "dr", "di", "dA_log", "dinit"], [x, r, i, A_log, init]
    if z is not None:
        names, leaves = ["dz"] + names, [z] + leaves
    return dict(zip(names, torch.autograd.grad(loss, leaves)))


def _exact_rotary(s):
    b, T, R, half = s["batch"], s["seqlen"], s["rotary"], s["rotary"] // 2
    place = torch.arange(T, device="cuda").expand(b, T) if s["positions"] is None else s["positions"]
    turn = torch.exp(1j * (place.double()[..., None, None] * s["freqs"]))
    out = {}
    for k in ("B", "C"):
        x, w = _leaf(s[k]), _leaf(s[k.lower() + "_weight"])
        v = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * w
        if s["interleaved"]:
            first, second = torch.arange(0, R, 2, device="cuda"), torch.arange(1, R, 2, device="cuda")
        else:
            first, second = torch.arange(half, device="cuda"), torch.arange(half, R, device="cuda")
        turned = torch.complex(v[..., first], v[..., second]) * turn
        rotated = v.index_copy(-1, first, turned.real).index_copy(-1, second, turned.imag)
        if s["pass"] == "forward":
            out[k] = rotated.detach()
        else:
            out["d" + k], out["d" + k.lower() + "_weight"] = torch.autograd.grad((rotated * s["d" + k]).sum(), (x, w))
    return out
