"""The operators of 4-bit experts, as they are measured: quantisation to 4 bits, the expert MLP of a few tokens
straight from the router's picks, and the ragged products grouped by expert (gate/up with SwiGLU, and down).

A 4-bit weight is w[e][n][k] = (q - z) * s with one scale s (bf16) and, where there are zero points, one z (0..15;
8 otherwise) for ``group`` consecutive columns of a row: q [E][n][k / 2] uint8, s and z [E][ceil(k / group)][n].
Eight columns of a row are one little-endian 32-bit word: nibble i (0..3) holds column 2 i, nibble 4 + i column
2 i + 1.
"""
import math

import torch

own = False

DEV = "cuda"

# The layer sizes of the repository's bench: decode and prefill d = 4096, 128 experts of 1536, top 8; block 256
# experts of 2048; tiny d = 256, 32 experts of 128.
_CASES = [
    # quantising a few small experts with zero points: odd sizes, a group that the columns do not fill
    dict(name="quantize_small", op="quantize", E=4, n=416, k=800, group=64, zero=True, x="bf16"),
    # quantising a stack of decode-sized expert matrices from fp32
    dict(name="quantize_experts", op="quantize", E=32, n=1536, k=4096, group=128, zero=False, x="f32"),
    # one token of the tiny layer in fp32: pure latency
    dict(name="picks_tiny", op="picks", T=1, d=256, E=32, f=128, top=8, group=32, zero=True, out="f32"),
    # one token of the decode layer: the single-user serving step
    dict(name="picks_one_token", op="picks", T=1, d=4096, E=128, f=1536, top=8, group=128, zero=False, out="bf16"),
    # a few tokens (a speculative step) of a layer with odd sizes
    dict(name="picks_five_tokens", op="picks", T=5, d=2080, E=48, f=992, top=3, group=64, zero=True, out="f32"),
    # a small serving batch of the decode layer
    dict(name="picks_sixteen_tokens", op="picks", T=16, d=4096, E=128, f=1536, top=8, group=128, zero=False, out="bf16"),
    # the decode workload's gate/up: about eight rows per expert
    dict(name="gate_up_decode", op="gate_up", T=128, d=4096, E=128, f=1536, top=8, group=128, zero=False, skew=0.0),
    # the decode workload's down with zero points and finer groups
    dict(name="down_decode", op="down", T=128, d=4096, E=128, f=1536, top=8, group=32, zero=True, skew=0.0),
    # a ragged chunk of a prompt through a layer with odd sizes, some experts hot and some empty
    dict(name="gate_up_ragged", op="gate_up", T=700, d=1888, E=24, f=1120, top=4, group=32, zero=True, skew=1.2),
    # the block workload's down: about 128 rows per expert
    dict(name="down_block", op="down", T=4096, d=4096, E=256, f=2048, top=8, group=64, zero=False, skew=0.0),
    # the prefill workload's gate/up: about 512 rows per expert
    dict(name="gate_up_prefill", op="gate_up", T=8192, d=4096, E=128, f=1536, top=8, group=128, zero=False, skew=0.5),
    # the prefill workload's down
    dict(name="down_prefill", op="down", T=8192, d=4096, E=128, f=1536, top=8, group=128, zero=True, skew=0.5),
]


def listed():
    return [dict(c) for c in _CASES]


def _log_int(rng, lo, hi, step=1):
    return max(lo, min(hi, step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)))


def draw(rng):
    op = rng.choice(["quantize", "picks", "picks", "gate_up", "gate_up", "down", "down"])
    group, zero = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "quantize":
        E, n = _log_int(rng, 1, 32), _log_int(rng, 32, 1536, 8)
        return dict(op=op, E=E, n=n, k=_log_int(rng, 32, 4096, 32), group=group, zero=zero, x=rng.choice(["bf16", "f32"]))
    d, f = _log_int(rng, 256, 4096, 32), _log_int(rng, 128, 1536, 32)
    E = _log_int(rng, 8, 128)
    top = rng.randint(1, 8)
    if op == "picks":
        return dict(op=op, T=_log_int(rng, 1, 16), d=d, E=E, f=f, top=top, group=group, zero=zero,
                    out=rng.choice(["bf16", "f32"]))
    return dict(op=op, T=_log_int(rng, 1, 8192), d=d, E=E, f=f, top=top, group=group, zero=zero,
                skew=rng.choice([0.0, 0.5, 1.2]))


# ------------------------------------------------------------------------------------------------ inputs
def _columns(k, group, zero, E, n, gen):
    """Scales and zero points of E matrices [n][k] whose weights have a variance of about 1 / k."""
    G = -(-k // group)
    s = (0.7 + 0.6 * torch.rand((E, G, n), generator=gen, device=DEV)) * (3.0 / 7.0) / math.sqrt(k)
    rest = (1 << (24 - (4 if zero else 5))) - 1  # the quantiser's scales have so few significant bits
    s = ((s.view(torch.int32) + rest) & ~rest).view(torch.float32).to(torch.bfloat16)
    z = torch.randint(5, 11, (E, G, n), generator=gen, device=DEV, dtype=torch.uint8) if zero else None
    return s, z


def _codes(E, n, k, gen):
    """Packed codes with the bell shape that quantised weights have."""
    q = torch.empty((E, n, k // 2), dtype=torch.uint8, device=DEV)
    for e in range(E):
        c = torch.randn((2, n, k // 2), generator=gen, device=DEV).mul_(2.4).add_(8.0).round_().clamp_(0, 15).to(torch.uint8)
        q[e] = c[0] | (c[1] << 4)
    return q


def _weights(E, n, k, group, zero, gen):
    s, z = _columns(k, group, zero, E, n, gen)
    return dict(q=_codes(E, n, k, gen), s=s, z=z, group=group, k=k)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    if c["op"] == "quantize":
        # trained weights: a normal bulk, rows of different spread, some columns pruned to zero
        W = torch.randn((c["E"], c["n"], c["k"]), generator=gen, device=DEV) / math.sqrt(c["k"])
        W *= 0.5 + torch.rand((c["E"], c["n"], 1), generator=gen, device=DEV)
        W[:, ::7, : min(c["k"], 128)] = 0
        return dict(c, W=W.to(torch.bfloat16) if c["x"] == "bf16" else W)
    T, d, E, f, top, group, zero = (c[n] for n in ("T", "d", "E", "f", "top", "group", "zero"))
    skew = c.get("skew", 0.0)
    # the router: distinct picks per token, popular experts first by a power law where there is skew
    pop = -skew * torch.log(torch.randperm(E, generator=gen, device=DEV).float() + 1)
    g = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device=DEV).clamp(1e-6, 1 - 1e-6)))
    score, idx = (pop + g).topk(top, dim=1)
    idx = idx.to(torch.int32)
    if c["op"] == "picks":
        w = torch.sigmoid(score)
        w = w / w.sum(1, keepdim=True)
        dt = torch.float32 if c["out"] == "f32" else torch.bfloat16
        st = dict(c, idx=idx, w=w, v=torch.randn((T, d), generator=gen, device=DEV).to(torch.bfloat16),
                  residual=torch.randn((T, d), generator=gen, device=DEV).to(dt),
                  gate=_weights(E, f, d, group, zero, gen), up=_weights(E, f, d, group, zero, gen),
                  down=_weights(E, d, f, group, zero, gen))
        return st
    counts = torch.bincount(idx.flatten(), minlength=E).to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    st = dict(c, counts=counts, offsets=offsets, rows=counts.tolist())
    S = T * top
    if c["op"] == "gate_up":
        st.update(x=torch.randn((S, d), generator=gen, device=DEV).to(torch.bfloat16),
                  gate=_weights(E, f, d, group, zero, gen), up=_weights(E, f, d, group, zero, gen))
    else:
        a = torch.randn((S, f), generator=gen, device=DEV)
        st.update(x=(a * torch.sigmoid(a) * torch.randn((S, f), generator=gen, device=DEV)).to(torch.bfloat16),
                  down=_weights(E, d, f, group, zero, gen))
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _unpack(q):
    """Codes [..., k] of packed bytes [..., k / 2]: low nibbles of a word's bytes hold columns 0, 4, 1, 5, high ones 2, 6, 3, 7."""
    b = q.reshape(*q.shape[:-1], -1, 4)
    c = torch.stack([b & 15, b >> 4], dim=-1).reshape(*b.shape[:-1], 8)  # columns 0, 2, 4, 6, 1, 3, 5, 7
    order = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=q.device)
    return c[..., order].reshape(*q.shape[:-1], -1)


def _plain_weight(w, e):
    """fp32 weights [..., n, k] of the experts e (an index or an index tensor)."""
    codes = _unpack(w["q"][e]).float()
    zero = w["z"][e].float() if w["z"] is not None else torch.full_like(w["s"][e], 8.0, dtype=torch.float32)
    s = w["s"][e].float()
    wide = lambda t: t.transpose(-1, -2).repeat_interleave(w["group"], dim=-1)[..., : w["k"]]  # noqa: E731
    return (codes - wide(zero)) * wide(s)


def _plain_quantize(st):
    W, group, zero = st["W"], st["group"], st["zero"]
    E, n, k = W.shape
    G = -(-k // group)
    x = torch.zeros((E, n, G * group), dtype=torch.float32, device=W.device)
    x[..., :k] = W.float()
    x = x.reshape(E, n, G, group)
    # 64 bits: where a scale or a code is rounded decides a whole step
    if zero:
        lo, hi = x.amin(-1).clamp(max=0).double(), x.amax(-1).clamp(min=0).double()
        t, steps, bits = hi - lo, 15.0, 4
    else:
        t, steps, bits = x.abs().amax(-1).double(), 7.0, 5
    t = t / torch.full_like(t, steps)  # a quotient: a division by a number may be a product with its reciprocal
    # up to the next number of so many significant bits, in the number's own bits
    rest = (1 << (53 - bits)) - 1
    s = ((t.view(torch.int64) + rest) & ~rest).view(torch.float64).clamp(min=2.0 ** -100)
    s = torch.where(t > 0, s, torch.ones_like(s))
    z = (-lo / s).round().clamp(0, 15) if zero else torch.full_like(s, 8.0)
    q = x.double().div_(s[..., None]).round_().add_(z[..., None]).clamp_(0, 15)
    values = ((q - z[..., None]) * s[..., None]).float().reshape(E, n, G * group)[..., :k].contiguous()
    return values, s.transpose(1, 2).to(torch.bfloat16).contiguous(), z.transpose(1, 2).to(torch.int32).contiguous()


def _plain_picks(st):
    e, x = st["idx"].long(), st["v"].float()[:, None, :, None]  # [T][top], [T][1][d][1]
    g = _plain_weight(st["gate"], e) @ x
    h = g / (1 + torch.exp(-g)) * (_plain_weight(st["up"], e) @ x)
    y = (_plain_weight(st["down"], e) @ h)[..., 0]  # [T][top][d]
    return (st["residual"].float() + (st["w"][..., None] * y).sum(1)).to(st["residual"].dtype)


def _plain_grouped(st):
    x = st["x"]
    n_out = st["f"] if st["op"] == "gate_up" else st["d"]
    out = torch.empty((x.shape[0], n_out), dtype=torch.bfloat16, device=x.device)
    at = 0
    for e, n in enumerate(st["rows"]):
        if n == 0:
            continue
        rows = x[at: at + n].float()
        if st["op"] == "gate_up":
            g = rows @ _plain_weight(st["gate"], e).T
            u = rows @ _plain_weight(st["up"], e).T
            out[at: at + n] = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
        else:
            out[at: at + n] = (rows @ _plain_weight(st["down"], e).T).to(torch.bfloat16)
        at += n
    return out


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    st = state
    if own:
        import moe_layer_forward_b200 as moe

        if st["op"] == "quantize":
            W4 = moe.quantize_w4_weights(st["W"], group=st["group"], zero=st["zero"])
            values = torch.empty(st["W"].shape, dtype=torch.float32, device=st["W"].device)
            moe.moe_dequantize_w4(W4, values)
            z = W4.z.int() if st["zero"] else torch.full(W4.s.shape, 8, dtype=torch.int32, device=values.device)
            return values, W4.s, z
        W4 = {n: moe.W4Weights(st[n]["q"], st[n]["s"], st[n]["z"], st["group"]) for n in ("gate", "up", "down") if n in st}
        if st["op"] == "picks":
            out = torch.empty_like(st["residual"])
            if "ws" not in st:
                n = moe.picks_w4_workspace_bytes(st["v"], W4["gate"], W4["down"], st["idx"])
                st["ws"] = torch.empty(n, dtype=torch.uint8, device=out.device)
            moe.moe_picks_swiglu_w4(st["v"], W4["gate"], W4["up"], W4["down"], st["idx"], st["w"], st["residual"], out,
                                    ws=st["ws"])
            return out
        x = st["x"]
        if st["op"] == "gate_up":
            h = torch.empty((x.shape[0], st["f"]), dtype=torch.bfloat16, device=x.device)
            moe.moe_expert_gate_up_w4(x, W4["gate"], W4["up"], st["counts"], st["offsets"], h)
            return h
        y = torch.empty((x.shape[0], st["d"]), dtype=torch.bfloat16, device=x.device)
        moe.moe_expert_down_w4(x, W4["down"], st["counts"], st["offsets"], y)
        return y
    if st["op"] == "quantize":
        return _plain_quantize(st)
    if st["op"] == "picks":
        return _plain_picks(st)
    return _plain_grouped(st)


# ------------------------------------------------------------------------------------------------ floors
def _stored(n, k, group, zero):
    return n * k / 2 + -(-k // group) * n * (3 if zero else 2)


def work(case):
    c = case
    if c["op"] == "quantize":
        size, G = c["E"] * c["n"] * c["k"], -(-c["k"] // c["group"])
        scales = c["E"] * c["n"] * G
        # the weights in, codes, scales and zero points kept, the values and the integer zero points out
        return {"bytes": size * (2 if c["x"] == "bf16" else 4) + 2 * _stored(c["E"] * c["n"], c["k"], c["group"], c["zero"])
                + 4 * size + 4 * scales, "flops": 4 * size}
    T, d, E, f, top, group, zero = (c[n] for n in ("T", "d", "E", "f", "top", "group", "zero"))
    S = T * top
    # experts that T tokens of `top` distinct picks reach (evenly routed: with skew a few less)
    active = E * (1 - (1 - top / E) ** T)
    up, down = active * _stored(f, d, group, zero), active * _stored(d, f, group, zero)
    if c["op"] == "picks":
        item = 4 if c["out"] == "f32" else 2
        return {"bytes": 2 * up + down + T * d * (2 + 2 * item) + 8 * S, "flops": 6 * S * d * f}
    if c["op"] == "gate_up":
        return {"bytes": 2 * up + 2 * S * d + 2 * S * f + 8 * E, "flops": 4 * S * d * f}
    return {"bytes": down + 2 * S * f + 2 * S * d + 8 * E, "flops": 2 * S * d * f}


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_matrix(w, e):
    """fp64 [n, k] of expert e, column by column of each word from the format's table."""
    q = w["q"][e]
    word = q.reshape(q.shape[0], -1, 4).long()
    word = word[..., 0] + (word[..., 1] << 8) + (word[..., 2] << 16) + (word[..., 3] << 24)
    out = torch.empty((q.shape[0], w["k"]), dtype=torch.float64, device=q.device)
    for j in range(8):
        nibble = (j // 2) + 4 * (j % 2)
        out[:, j::8] = ((word >> (4 * nibble)) & 15).double()
    group_of = torch.arange(w["k"], device=q.device) // w["group"]
    out -= w["z"][e].double()[group_of].T if w["z"] is not None else 8.0
    return out.mul_(w["s"][e].double()[group_of].T)


def _exact_quantize(st):
    W, group = st["W"], st["group"]
    E, n, k = W.shape
    G = -(-k // group)
    values = torch.empty((E, n, k), dtype=torch.float64, device=W.device)
    scales = torch.empty((E, G, n), dtype=torch.float64, device=W.device)
    zeros = torch.full((E, G, n), 8, dtype=torch.int32, device=W.device)
    for j in range(G):
        x = W[..., j * group: (j + 1) * group].double()
        if st["zero"]:
            lo = torch.minimum(x.min(-1).values, torch.zeros((), dtype=torch.float64, device=W.device))
            least = torch.maximum(x.max(-1).values, torch.zeros_like(lo)) - lo
            least, bits = least / torch.full_like(least, 15.0), 4
        else:
            lo, least, bits = None, x.abs().max(-1).values, 5
            least = least / torch.full_like(least, 7.0)
        live = least > 0
        binade = ((least.view(torch.int64) >> 52) << 52).view(torch.float64)  # 2^floor(log2 least)
        unit = torch.where(live, binade, torch.ones_like(binade)) * 2.0 ** (1 - bits)
        s = torch.where(live, torch.ceil(least / unit) * unit, torch.ones_like(least))
        s = torch.maximum(s, torch.full_like(s, 2.0 ** -100))
        if st["zero"]:
            z = torch.clamp(torch.round(-lo / s), 0, 15)
            zeros[:, j] = z.int()
            code = torch.clamp(torch.round(x / s[..., None]), -z[..., None], 15 - z[..., None])
        else:
            code = torch.clamp(torch.round(x / s[..., None]), -8, 7)
        values[..., j * group: (j + 1) * group] = code * s[..., None]
        scales[:, j] = s
    return values, scales, zeros


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "quantize":
        return _exact_quantize(st)
    silu = lambda g: g * torch.sigmoid(g)  # noqa: E731
    if st["op"] == "picks":
        out = st["residual"].double()
        for e in st["idx"].unique().tolist():
            token, pick = torch.nonzero(st["idx"] == e, as_tuple=True)
            v = st["v"].double()[token]
            h = silu(v @ _exact_matrix(st["gate"], e).T) * (v @ _exact_matrix(st["up"], e).T)
            out.index_add_(0, token, st["w"].double()[token, pick][:, None] * (h @ _exact_matrix(st["down"], e).T))
        return out
    bounds = st["offsets"].tolist()
    parts = []
    for e in range(st["E"]):
        x = st["x"][bounds[e]: bounds[e + 1]].double()
        if x.shape[0] == 0:
            continue
        if st["op"] == "gate_up":
            parts.append(silu(x @ _exact_matrix(st["gate"], e).T) * (x @ _exact_matrix(st["up"], e).T))
        else:
            parts.append(x @ _exact_matrix(st["down"], e).T)
    return torch.cat(parts)
