"""The serving step of a block-diffusion model over a KV cache held in 8 bits, operator by operator.

One decoding step of a block of b tokens rotates the block's queries and keys (rotary positions),
quantises its keys and values into the cache as it writes them, attends to the cache as it is held,
and verifies the drafted block against the target's probabilities; the rotation and its gradient
also stand on both sides of the training form's attention.  Each case below is one call.

``run`` computes a case in its plain form, with elementary torch operations in 32 bits (64 for
angles and for the sums and comparisons of the verification), or, with ``own``, by the calls that a
user of the package makes.  Cache lengths and accepted counts follow from the case alone, so that
``work`` is exact; every value follows from the seed.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -64  # the smallest scale is 2^-64


# ----------------------------------------------------------------------------
# cases


def _rope(name, B, Hq, Hkv, rows, d, rot, interleaved=False, adjoint=False, factor=1.0, lo=0, hi=0):
    """rows > 0 with hi > 0: a decoded block of that many rows at cache lengths lo..hi.  hi = 0: the training form [x_t ; x_0] of rows + rows tokens."""
    return dict(name=name, op="rope", B=B, Hq=Hq, Hkv=Hkv, rows=rows, d=d, rot=rot, interleaved=interleaved, adjoint=adjoint, factor=factor, lo=lo, hi=hi)


def _append(name, B, Hkv, rows, d, group, lo, hi, ragged):
    """rows new rows a sequence (with ragged: 0..rows of them) behind lo..hi cached ones."""
    return dict(name=name, op="append", B=B, Hkv=Hkv, rows=rows, d=d, group=group, lo=lo, hi=hi, ragged=ragged)


def _read(name, B, Hkv, d, group, lo, hi):
    return dict(name=name, op="read", B=B, Hkv=Hkv, d=d, group=group, lo=lo, hi=hi)


def _decode(name, B, Hq, Hkv, rows, d, group, mode, lo, hi):
    """rows queries a sequence over lo..hi cached rows; mode 0 bidirectional in the block, 1 causal, 2 the prefix alone."""
    return dict(name=name, op="decode", B=B, Hq=Hq, Hkv=Hkv, rows=rows, d=d, group=group, mode=mode, lo=lo, hi=hi)


def _verify(name, B, rows, V, point):
    """rows drafted tokens a sequence over a vocabulary of V; point: the draft was taken greedily and has no probabilities."""
    return dict(name=name, op="verify", B=B, rows=rows, V=V, point=point)


def listed():
    return [
        # the queries and keys of a denoised block, every step and layer: latency
        _rope("rope block", 16, 32, 8, 32, 128, 128, lo=8192, hi=8192),
        # the training shape's queries and keys before attention, noisy and clean tokens at the same positions
        _rope("rope train", 4, 32, 8, 2048, 128, 128),
        # the gradient of a rotation of half of a smaller head, pairs side by side, frequencies scaled for a long context
        _rope("rope train gradient", 3, 8, 2, 4099, 64, 32, interleaved=True, adjoint=True, factor=8.0),
        # the accepted rows of a verified block behind ragged prefixes, every step and layer: latency
        _append("append accepted", 64, 8, 28, 128, 64, 512, 8192, True),
        # a prompt's keys and values on their way into an empty cache
        _append("append prompt", 4, 8, 8192, 128, 128, 0, 0, False),
        # the prefix back in 16 bits, as pruning it needs
        _read("read back", 16, 8, 128, 64, 4001, 8192),
        # one token of one short sequence: the smallest call
        _decode("decode one token", 1, 8, 2, 1, 64, 32, 1, 777, 777),
        # single tokens of a batch over long prefixes
        _decode("decode tokens", 24, 32, 8, 1, 128, 128, 1, 4096, 32768),
        # a block denoised over full prefixes
        _decode("decode denoise", 16, 32, 8, 32, 128, 64, 0, 8192, 8192),
        # drafted blocks verified over ragged prefixes
        _decode("decode verify", 64, 32, 8, 28, 128, 64, 1, 512, 8192),
        # one drafted block of one sequence over an odd vocabulary
        _verify("verify one", 1, 28, 50001, False),
        # drafted blocks of a batch over a large vocabulary
        _verify("verify batch", 64, 28, 131072, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode", "decode", "verify"])
    d = rng.choice([32, 64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    B = _log(rng, 1, 64)
    group = rng.choice([16, 32, 64, 128])
    if op == "rope":
        Hq = Hkv * rng.choice([1, 2, 4])
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
        two = dict(interleaved=rng.random() < 0.5, adjoint=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 8.0, 32.0]))
        if rng.random() < 0.5:
            lo = _log(rng, 1, 100000)
            return {k: v for k, v in _rope("", B, Hq, Hkv, _log(rng, 1, 64), d, rot, lo=lo, hi=lo + _log(rng, 1, 100000), **two).items() if k != "name"}
        most = max(2, 4 * 40 * 2048 * 128 // (B * (Hq + Hkv) * d))
        return {k: v for k, v in _rope("", B, Hq, Hkv, _log(rng, 1, min(8192, most)), d, rot, **two).items() if k != "name"}
    if op == "append":
        rows = _log(rng, 1, max(2, min(8192, 4 * 8 * 8192 * 128 // (B * Hkv * d))))
        lo = rng.choice([0, _log(rng, 1, 4096)])
        return {k: v for k, v in _append("", B, Hkv, rows, d, group, lo, lo + rng.randrange(4096), rng.random() < 0.5).items() if k != "name"}
    if op == "read":
        hi = _log(rng, 1, max(2, min(16384, 16 * 8 * 6096 * 128 // (B * Hkv * d))))
        return {k: v for k, v in _read("", B, Hkv, d, group, rng.randrange(hi + 1), hi).items() if k != "name"}
    if op == "decode":
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        rows = _log(rng, 1, 64)
        mode = rng.choice([0, 1, 1, 2])
        hi = _log(rng, 8, max(16, min(32768, 16 * 32 * 32 * 8192 * 128 // (B * Hq * rows * d), 64 * 8 * 4096 * 128 // (B * Hkv * d))))
        return {k: v for k, v in _decode("", B, Hq, Hkv, rows, d, group, mode, rng.randrange(1, hi + 1), hi).items() if k != "name"}
    V = _log(rng, 100, 131072)
    return {k: v for k, v in _verify("", B, rng.randrange(1, 29), V, rng.random() < 0.3).items() if k != "name"}


def _spread(n, lo, hi):
    """n whole numbers spread over lo..hi, the same ones for the same case."""
    return [lo + (i * 2654435761 + 12345) % 4294967296 % (hi - lo + 1) for i in range(n)]


def _capacity(case, lens, own_rows):
    g = case["group"]
    return -(-(max(lens) + own_rows) // g) * g + g


def _counts(case):
    return _spread(case["B"], 0, case["rows"]) if case["ragged"] else [case["rows"]] * case["B"]


# ----------------------------------------------------------------------------
# inputs


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _inv_freq(rot, factor, base=10000.0, trained=4096, fast=32.0, slow=1.0):
    """Frequencies of the pairs in radians a position, 64 bits: with a factor over 1, pairs that turn more than `fast` times over the trained length stay, pairs that turn less than `slow` times are slowed by the factor, the rest in between."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = base ** (-2.0 * i / rot)
    keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
    return f / factor * (1 - keep) + f * keep


def _scales(x, group):
    """The smallest power of two, 2^-64 or more, that holds each group's largest value within +-448, for rows a multiple of the group."""
    B, H, S, d = x.shape
    m, e = torch.frexp(x.float().reshape(B, H, S // group, group * d).abs().amax(-1))
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=MIN_EXP)
    k = torch.where(m == 0, torch.full_like(k, MIN_EXP), k)
    return torch.ldexp(torch.ones_like(m), k)


def _quantised(g, B, H, S, d, group):
    """A cache as earlier steps wrote it: heads of different magnitude, groups with their own scales."""
    x = _randn(g, B, H, S, d) * torch.exp2(torch.randint(-2, 3, (B, H, 1, 1), generator=g, device="cuda").float())
    s = _scales(x, group)
    return (x / s.repeat_interleave(group, 2).unsqueeze(-1)).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g, op, B = _gen(seed), case["op"], case["B"]
    s = dict(case)
    if op == "rope":
        block = case["hi"] > 0
        n = case["rows"] if block else 2 * case["rows"]
        s["q"] = _randn(g, B, case["Hq"], n, case["d"]).to(torch.bfloat16)
        s["k"] = _randn(g, B, case["Hkv"], n, case["d"]).to(torch.bfloat16)
        s["start"] = _int32(_spread(B, case["lo"], case["hi"])) if block else None
        s["inv_freq"] = _inv_freq(case["rot"], case["factor"])
        s["mscale"] = 0.1 * math.log(case["factor"]) + 1.0
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        return s
    if op == "verify":
        V, n = case["V"], case["rows"]
        z = _randn(g, B, n + 1, V)
        s["target_prob"] = torch.softmax(2.0 * z + 0.7 * _randn(g, B, n + 1, V), -1)
        q = torch.softmax(2.0 * z[:, :n], -1)
        if case["point"]:
            s["draft"], s["draft_prob"] = q.argmax(-1).to(torch.int32), None
        else:
            s["draft"] = torch.multinomial(q.reshape(B * n, V), 1, generator=g).reshape(B, n).to(torch.int32)
            s["draft_prob"] = q
        s["u_accept"] = torch.rand((B, n), generator=g, device="cuda")
        s["u_sample"] = torch.rand((B,), generator=g, device="cuda")
        s["n_accept"], s["next_token"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
        return s
    Hkv, d, group = case["Hkv"], case["d"], case["group"]
    lens = _spread(B, case["lo"], case["hi"])
    rows = case["rows"] if op == "append" or (op == "decode" and case["mode"] != 2) else 0
    S = _capacity(case, lens, rows)
    s["k_cache"], s["k_scale"] = _quantised(g, B, Hkv, S, d, group)
    s["v_cache"], s["v_scale"] = _quantised(g, B, Hkv, S, d, group)
    s["cache_len"] = _int32(lens)
    if op == "append":
        s["k_new"] = (2.0 * _randn(g, B, Hkv, rows, d)).to(torch.bfloat16)
        s["v_new"] = _randn(g, B, Hkv, rows, d).to(torch.bfloat16)
        s["n_new"] = _int32(_counts(case)) if case["ragged"] else None
    elif op == "read":
        s["k_out"], s["v_out"] = (torch.zeros((B, Hkv, S, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        s["q"] = _randn(g, B, case["Hq"], case["rows"], d).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, case["Hq"], case["rows"]), device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _run_own(s)
    return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "decode": _plain_decode, "verify": _plain_verify}[s["op"]](s)


def _run_own(s):
    import block_diffusion_lm_attn_b200 as bd
    op = s["op"]
    if op == "rope":
        return bd.rope(s["q"], s["k"], s["inv_freq"], start=s["start"], period=s["rows"], interleaved=s["interleaved"], mscale=s["mscale"], adjoint=s["adjoint"], q_out=s["q_out"], k_out=s["k_out"])
    if op == "append":
        bd.cache_append_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["cache_len"], s["k_new"], s["v_new"], s["group"], n_new=s["n_new"], advance=False)
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "read":
        return bd.cache_read_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["cache_len"], s["group"], k_out=s["k_out"], v_out=s["v_out"])
    if op == "decode":
        return bd.decode_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["cache_len"], s["mode"], s["group"], out=s["out"], lse=s["lse"])
    return bd.spec_verify(s["draft"], s["draft_prob"], s["target_prob"], s["u_accept"], s["u_sample"], n_accept=s["n_accept"], next_token=s["next_token"])


def _plain_rope(s):
    n, rot = s["q"].shape[2], s["rot"]
    pos = torch.arange(n, device="cuda") % s["rows"]
    pos = pos[None] if s["start"] is None else pos[None] + s["start"][:, None]
    angle = pos[:, None, :, None].double() * s["inv_freq"]
    c, t = (s["mscale"] * angle.cos()).float(), (s["mscale"] * angle.sin()).float()
    t = -t if s["adjoint"] else t

    def turn(x):
        x = x.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., : rot // 2], x[..., rot // 2 : rot])
        a, b = a * c - b * t, b * c + a * t
        y = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((y, x[..., rot:]), -1).to(torch.bfloat16)

    return turn(s["q"]), turn(s["k"])


def _plain_append(s):
    B, H, S, d = s["k_cache"].shape
    group, rows = s["group"], s["rows"]
    n = s["n_new"][:, None] if s["n_new"] is not None else rows
    length = s["cache_len"][:, None].long()
    width = min(S, (-(-rows // group) + 1) * group)  # the groups that the new rows can touch
    at = (length // group * group).clamp(max=S - width) + torch.arange(width, device="cuda")
    new = (at >= length) & (at < length + n)
    keep = at < length
    touched = new.reshape(B, -1, group).any(-1)
    rows_at = at[:, None, :, None].expand(B, H, width, d)
    from_at = (at - length).clamp(0, rows - 1)[:, None, :, None].expand(B, H, width, d)
    groups_at = at[:, None, ::group].expand(B, H, width // group) // group
    for x, cache, scale in ((s["k_new"], s["k_cache"], s["k_scale"]), (s["v_new"], s["v_cache"], s["v_scale"])):
        codes = cache.view(torch.uint8)
        old = codes.gather(2, rows_at)
        old_scale = scale.gather(2, groups_at)
        value = old.view(torch.float8_e4m3fn).float() * old_scale.repeat_interleave(group, 2).unsqueeze(-1)
        value = torch.where(keep[:, None, :, None], value, torch.zeros_like(value))
        value = torch.where(new[:, None, :, None], x.gather(2, from_at).float(), value)
        to = torch.where(touched[:, None], _scales(value, group), old_scale)
        code = (value / to.repeat_interleave(group, 2).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        write = (touched.repeat_interleave(group, 1) & (new | keep))[:, None, :, None]
        codes.scatter_(2, rows_at, torch.where(write, code.view(torch.uint8), old))
        scale.scatter_(2, groups_at, to)
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_read(s):
    live = (torch.arange(s["k_cache"].shape[2], device="cuda") < s["cache_len"][:, None])[:, None, :, None]
    for cache, scale, out in ((s["k_cache"], s["k_scale"], s["k_out"]), (s["v_cache"], s["v_scale"], s["v_out"])):
        x = cache.float() * scale.repeat_interleave(s["group"], 2).unsqueeze(-1)
        out.copy_(torch.where(live, x.to(torch.bfloat16), out))
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    B, Hq, b, d = s["q"].shape
    _, H, S, _ = s["k_cache"].shape
    own_rows = (b, 1, 0)[s["mode"]]
    rows = torch.arange(b, device="cuda") if s["mode"] == 1 else torch.zeros(b, dtype=torch.long, device="cuda")
    seen = s["cache_len"][:, None] + own_rows + rows  # keys that row j of a sequence sees
    k = s["k_cache"].float() * s["k_scale"].repeat_interleave(s["group"], 2).unsqueeze(-1)
    v = s["v_cache"].float() * s["v_scale"].repeat_interleave(s["group"], 2).unsqueeze(-1)
    q = s["q"].float().reshape(B, H, Hq // H * b, d)
    x = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    mask = torch.arange(S, device="cuda") < seen.repeat(1, Hq // H)[:, None, :, None]
    x = torch.where(mask, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / l
    return out.reshape(B, Hq, b, d).to(torch.bfloat16), (m + torch.log(l)).reshape(B, Hq, b)


def _plain_verify(s):
    B, n = s["draft"].shape
    token = s["draft"].long().unsqueeze(-1)
    p = s["target_prob"][:, :n].gather(2, token).squeeze(-1).double()
    q = s["draft_prob"].gather(2, token).squeeze(-1).double() if s["draft_prob"] is not None else torch.ones_like(p)
    accepted = torch.cumprod((s["u_accept"].double() * q < p).to(torch.int32), 1).sum(1)
    row = torch.arange(B, device="cuda")
    at = accepted.clamp(max=n - 1)
    p = s["target_prob"][row, accepted].double()
    if s["draft_prob"] is not None:
        q = s["draft_prob"][row, at].double()
    else:
        q = torch.zeros_like(p).scatter_(1, s["draft"][row, at].long().unsqueeze(-1), 1.0)
    w = torch.where((accepted < n).unsqueeze(-1), p - q, p).clamp(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    c = w.cumsum(1)
    first = (c <= s["u_sample"].double().unsqueeze(-1) * c[:, -1:]).sum(1)
    last = c.shape[1] - 1 - (w > 0).flip(1).to(torch.int32).argmax(1)
    return accepted.to(torch.int32), torch.minimum(first, last).to(torch.int32)


# ----------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, B = case["op"], case["B"]
    if op == "rope":
        n = case["rows"] if case["hi"] > 0 else 2 * case["rows"]
        values = B * (case["Hq"] + case["Hkv"]) * n
        return {"bytes": 4.0 * values * case["d"], "flops": 3.0 * values * case["rot"]}
    if op == "verify":
        # the row at the first refusal: the target's, and the draft's where it has one
        return {"bytes": 4.0 * B * (case["V"] * (1 if case["point"] else 2) + 5 * case["rows"]), "flops": 4.0 * B * case["V"]}
    Hkv, d, group = case["Hkv"], case["d"], case["group"]
    lens = _spread(B, case["lo"], case["hi"])
    if op == "append":
        new = sum(_counts(case))
        # the rows that share the first group with the new ones are read and written again
        old = sum(a % group for a, c in zip(lens, _counts(case)) if c)
        groups = sum((a + c - 1) // group - a // group + 1 for a, c in zip(lens, _counts(case)) if c)
        return {"bytes": 2.0 * Hkv * (d * (3 * new + 2 * old) + 8 * groups), "flops": 4.0 * Hkv * d * (new + old)}
    if op == "read":
        return {"bytes": 2.0 * Hkv * sum(3 * d * a + 4 * -(-a // group) for a in lens), "flops": 2.0 * Hkv * d * sum(lens)}
    Hq, b = case["Hq"], case["rows"]
    keys = [a + (b if case["mode"] != 2 else 0) for a in lens]
    seen = sum({0: b * (a + b), 1: b * a + b * (b + 1) // 2, 2: b * a}[case["mode"]] for a in lens)
    cache = 2.0 * Hkv * sum(d * a + 4 * -(-a // group) for a in keys)
    return {"bytes": cache + 4.0 * B * Hq * b * d + 4.0 * B * Hq * b, "flops": 4.0 * Hq * d * seen}


# ----------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "read": _exact_read, "decode": _exact_decode, "verify": _exact_verify}[case["op"]](s)


def _exact_rope(s):
    """Each pair is a complex number, turned by e^(i angle) and stretched by mscale."""
    B, _, n, d = s["q"].shape
    rot = s["rot"]
    first = s["start"].tolist() if s["start"] is not None else [0] * B
    pos = torch.tensor([[f + r % s["rows"] for r in range(n)] for f in first], dtype=torch.float64, device="cuda")
    sign = -1.0 if s["adjoint"] else 1.0
    turn = torch.polar(torch.full((B, n, rot // 2), s["mscale"], dtype=torch.float64, device="cuda"), sign * pos.unsqueeze(-1) * s["inv_freq"])
    outs = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        if s["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * turn[:, None]
            y[..., :rot] = torch.view_as_real(z).reshape(*y.shape[:-1], rot)
        else:
            z = torch.complex(y[..., : rot // 2].contiguous(), y[..., rot // 2 : rot].contiguous()) * turn[:, None]
            y[..., : rot // 2], y[..., rot // 2 : rot] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _round_e4m3(x):
    """The nearest value of 1 + 4 + 3 bits, ties to even: steps of 2^-3 of the power of two below x, 2^-9 at least."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (x / step).round() * step


def _exact_append(s):
    group = s["group"]
    lens = s["cache_len"].tolist()
    counts = s["n_new"].tolist() if s["n_new"] is not None else [s["rows"]] * len(lens)
    outs = []
    for x, cache, scale in ((s["k_new"], s["k_cache"], s["k_scale"]), (s["v_new"], s["v_cache"], s["v_scale"])):
        codes, scales = cache.float().double(), scale.double()
        for i, (a, c) in enumerate(zip(lens, counts)):
            if c == 0:
                continue
            g0, g1 = a // group, (a + c - 1) // group + 1
            value = torch.zeros_like(codes[i, :, g0 * group : g1 * group])
            old = a - g0 * group
            value[:, :old] = codes[i, :, g0 * group : a] * scales[i, :, g0, None, None]
            value[:, old : old + c] = x[i, :, :c].double()
            top = value.reshape(value.shape[0], g1 - g0, -1).abs().amax(-1)
            power = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=MIN_EXP)
            power = torch.where(top > E4M3_MAX * torch.exp2(power), power + 1, power)
            power = torch.where((top <= E4M3_MAX * torch.exp2(power - 1)) & (power > MIN_EXP), power - 1, power)
            to = torch.exp2(power)
            scales[i, :, g0:g1] = to
            codes[i, :, g0 * group : a + c] = _round_e4m3(value / to.repeat_interleave(group, 1).unsqueeze(-1))[:, : old + c]
        outs.append((codes, scales))
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


def _exact_read(s):
    outs = []
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        y = torch.zeros(cache.shape, dtype=torch.float64, device="cuda")
        for i, a in enumerate(s["cache_len"].tolist()):
            y[i, :, :a] = cache[i, :, :a].float().double() * scale[i].double().repeat_interleave(s["group"], 1)[:, :a, None]
        outs.append(y)
    return tuple(outs)


def _exact_decode(s):
    B, Hq, b, d = s["q"].shape
    H = s["k_cache"].shape[1]
    out = torch.zeros((B, Hq, b, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, b), dtype=torch.float64, device="cuda")
    for i, a in enumerate(s["cache_len"].tolist()):
        n = a + (b if s["mode"] != 2 else 0)
        hidden = torch.zeros((b, n), dtype=torch.bool, device="cuda")
        if s["mode"] == 1:
            hidden[:, a:] = torch.ones((b, b), dtype=torch.bool, device="cuda").triu(1)
        for h in range(H):
            k, v = (c[i, h, :n].float().double() * z[i, h].double().repeat_interleave(s["group"])[:n, None] for c, z in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            mine = slice(h * (Hq // H), (h + 1) * (Hq // H))
            x = (s["q"][i, mine].double() @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[i, mine] = torch.logsumexp(x, -1)
            out[i, mine] = torch.exp(x - lse[i, mine].unsqueeze(-1)) @ v
    return out, lse


def _exact_verify(s):
    B, n = s["draft"].shape
    counts, tokens = [], []
    draft, u, r = s["draft"].tolist(), s["u_accept"].double().tolist(), s["u_sample"].double().tolist()
    for i in range(B):
        j = 0
        while j < n:
            q = s["draft_prob"][i, j, draft[i][j]].item() if s["draft_prob"] is not None else 1.0
            if not u[i][j] * q < s["target_prob"][i, j, draft[i][j]].item():
                break
            j += 1
        w = s["target_prob"][i, j].double().cpu().numpy().copy()
        if j < n:
            rest = w.copy()
            if s["draft_prob"] is not None:
                rest -= s["draft_prob"][i, j].double().cpu().numpy()
            else:
                rest[draft[i][j]] -= 1.0
            rest[rest < 0] = 0
            w = rest if rest.sum() > 0 else w
        c = w.cumsum()
        counts.append(j)
        tokens.append(int((c > r[i] * c[-1]).argmax()))
    return _int32(counts), _int32(tokens)
