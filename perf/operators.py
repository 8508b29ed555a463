"""Cases of the 8-bit KV cache and shared-prefix operators: what each takes, its
plain form in elementary torch operations, and its definition in 64 bits.

Five operators of a decode server:

write    a chunk of new keys and values (a prefill, or a chunk of one) is
         quantised into the 8-bit cache at each sequence's next slots;
read     rows of the 8-bit cache are read back as a bf16 cache;
append   one decode token per sequence: RoPE, quantised append, position-0
         capture, routing;
decode   routed split-K attention of one token over the 8-bit cache;
prefix   one token of every sequence of a batch over a prefix that all of them
         share (bf16, read once for all), joined with each sequence's own
         suffix where the case has one.

Shapes are the repository's workloads: Llama-3.1-8B (32 query / 8 KV heads, here
hkv=8, m=4), Llama-3.1-70B (hkv=8, m=8), LLaVA-1.5-7B (MHA: hkv=32, m=1),
head_dim 128. Which (sequence, group) units are sinks, and the ragged lengths,
follow from the case alone; every value follows from the seed.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"
TAU = 0.6
FLOOR = 2.0 ** -100  # a row's largest magnitude counts as at least this
LOG_BASE = math.log(500000.0)


# ---- cases -----------------------------------------------------------------------------

def listed():
    return [
        # A whole 128K prompt of the 8B-shaped layer is written after its prefill.
        dict(name="write_8b_prompt_128k_e4m3", op="write", kv="e4m3", b=1, hkv=8, t=131072, lmax=131072, ragged=False,
             fused=False),
        # Chunked prefill of four sequences: ragged chunk lengths and starts, k and v
        # as strided views of one fused projection, an odd capacity.
        dict(name="write_70b_chunk_ragged_int8", op="write", kv="int8", b=4, hkv=8, t=1021, lmax=8191, ragged=True,
             fused=True),
        # A 32K context leaves the 8-bit cache for the bf16 path.
        dict(name="read_8b_32k_int8", op="read", kv="int8", b=1, hkv=8, t=32768, lmax=32768, ragged=False),
        # The image tokens and a short prompt of eight MHA sequences, from odd starts.
        dict(name="read_llava_ragged_e4m3", op="read", kv="e4m3", b=8, hkv=32, t=577, lmax=2047, ragged=True),
        # One sequence decodes: latency.
        dict(name="append_8b_b1_e4m3", op="append", kv="e4m3", b=1, hkv=8, m=4, lmax=4096, sinks=4),
        # A full decode batch.
        dict(name="append_70b_b64_int8", op="append", kv="int8", b=64, hkv=8, m=8, lmax=513, sinks=3),
        # Short context: latency.
        dict(name="decode_8b_4k_e4m3", op="decode", kv="e4m3", b=1, hkv=8, m=4, lmax=4096, ragged=False, sinks=4),
        # The headline layer, half of its groups sinks.
        dict(name="decode_8b_128k_e4m3", op="decode", kv="e4m3", b=1, hkv=8, m=4, lmax=131072, ragged=False, sinks=4),
        # Four ragged 64K..128K contexts with eight heads a group.
        dict(name="decode_70b_ragged_128k_int8", op="decode", kv="int8", b=4, hkv=8, m=8, lmax=131072, ragged=True,
             sinks=3),
        # Eight samples of one 128K document, each with a short 8-bit suffix of its own: the prefix read is the bound.
        dict(name="prefix_8b_b8_128k_e4m3", op="prefix", kv="e4m3", b=8, hkv=8, m=4, lp=131072, lmax=512, sinks=2),
        # A serving batch over one 32K document, bf16 suffixes of up to 250 tokens: bound by arithmetic.
        dict(name="prefix_70b_b128_32k_bf16", op="prefix", kv="bf16", b=128, hkv=8, m=8, lp=32768, lmax=250, sinks=1),
        # The image tokens alone, shared by three MHA sequences, no suffix yet: latency, odd sizes.
        dict(name="prefix_llava_b3_577", op="prefix", kv="none", b=3, hkv=32, m=1, lp=577, lmax=0, sinks=3),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["write", "read", "append", "decode", "decode", "prefix", "prefix"])
    hkv, m = rng.choice([(8, 4), (8, 8), (32, 1), (4, 2), (5, 4)])
    kv = rng.choice(["e4m3", "int8"])
    if op in ("write", "read"):
        b = _log_int(rng, 1, 32)
        t = _log_int(rng, 1, max(1, 1048576 // (b * hkv)))
        c = dict(op=op, kv=kv, b=b, hkv=hkv, t=t, lmax=t + _log_int(rng, 1, max(1, t)), ragged=rng.random() < 0.6)
        if op == "write":
            c["fused"] = rng.random() < 0.5
        return c
    sinks = rng.randint(0, 7)
    if op == "append":
        b = _log_int(rng, 1, 128)
        return dict(op=op, kv=kv, b=b, hkv=hkv, m=m, lmax=_log_int(rng, 1, 2000), sinks=sinks)
    if op == "decode":
        b = _log_int(rng, 1, 64)
        return dict(op=op, kv=kv, b=b, hkv=hkv, m=m, lmax=_log_int(rng, 1, 2000000 // (b * hkv)),
                    ragged=rng.random() < 0.6, sinks=sinks)
    kv = rng.choice(["e4m3", "int8", "bf16", "none"])
    b = _log_int(rng, 1, 128)
    lp = _log_int(rng, 1, min(131072, 1048576 // hkv, 200000000 // (b * hkv * m)))
    lmax = 0 if kv == "none" else _log_int(rng, 1, min(2000, 400000 // (b * hkv)))
    return dict(op=op, kv=kv, b=b, hkv=hkv, m=m, lp=lp, lmax=lmax, sinks=sinks)


def _spread(n, lo, hi, step):
    """n lengths of [lo, hi], the first of them hi, the same for every seed."""
    return [hi - (i * step) % (hi - lo + 1) for i in range(n)]


def _counts(c):
    """(start, count) of every sequence's rows in a write or read."""
    b, t = c["b"], c["t"]
    n = _spread(b, t // 2, t, 7919) if c["ragged"] else [t] * b
    s = [(i * 613) % (c["lmax"] - t + 1) for i in range(b)] if c["ragged"] else [0] * b
    return s, n


def _lens(c):
    """Valid positions of every sequence's own cache."""
    if c["op"] == "decode" and not c["ragged"]:
        return [c["lmax"]] * c["b"]
    return _spread(c["b"], max(1, c["lmax"] // 2), c["lmax"], 7919)


def _sinks(c):
    """[b, hkv]: which units' queries point along the position-0 key."""
    b, g = np.arange(c["b"])[:, None], np.arange(c["hkv"])[None, :]
    return (5 * b + 3 * g) % 8 < c["sinks"]


def work(case):
    c = case
    hkv = c["hkv"]
    row8, row16 = D + 4, 2 * D  # bytes of a key or value row: 8-bit codes and a scale, or bf16
    if c["op"] in ("write", "read"):
        rows = 2 * sum(_counts(c)[1]) * hkv
        return {"bytes": rows * (row8 + row16), "flops": 3 * rows * D}
    b, hq = c["b"], hkv * c["m"]
    active = int((~_sinks(c)).sum(1).sum())
    qo = 2 * b * hq * row16
    small = 2 * b * hkv * row16  # k0 / v0 or the new key and value
    if c["op"] == "append":
        return {"bytes": qo + small + 2 * b * hkv * row8 + b * hkv * row16, "flops": (b * hq + b * hkv) * 3 * D + b * hq * 2 * D}
    per = (~_sinks(c)).sum(1)  # active groups of each sequence
    own_rows = 0 if c["op"] == "prefix" and c["kv"] == "none" else int((per * np.array(_lens(c))).sum())
    row = row16 if c["kv"] == "bf16" else row8
    need = {"bytes": qo + small + 2 * own_rows * row, "flops": 4 * own_rows * c["m"] * D}
    if c["op"] == "prefix":
        groups = int((~_sinks(c)).any(0).sum())
        need["bytes"] += 2 * groups * c["lp"] * row16
        need["flops"] += 4 * active * c["m"] * c["lp"] * D
    return need


# ---- inputs ----------------------------------------------------------------------------

def _gen(seed, role):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + role)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rows(shape, g):
    """bf16 rows as a trained projection leaves them: normal values, the rows' sizes spread over a factor of four."""
    x = torch.randn(shape, generator=g, device=DEV)
    return (x * (0.5 + 1.5 * torch.rand((*shape[:-1], 1), generator=g, device=DEV))).to(torch.bfloat16)


def _tables(n):
    inv = torch.exp(-LOG_BASE * torch.arange(0, D, 2, dtype=torch.float64) / D)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cos(ang).float().to(DEV), torch.sin(ang).float().to(DEV)


def _queries(c, k0, g):
    """Sink units: every head near the position-0 key. Others: heads with a cosine to it inside (-0.2, 0.2)."""
    m = c["m"]
    k = k0.float().repeat_interleave(m, 1)
    hat = k / k.norm(dim=-1, keepdim=True)
    r = torch.randn(k.shape, generator=g, device=DEV)
    r = r - (r * hat).sum(-1, keepdim=True) * hat
    tilt = (torch.rand((*k.shape[:2], 1), generator=g, device=DEV) * 2 - 1) * 0.2
    active = r + tilt * r.norm(dim=-1, keepdim=True) * hat
    near = k + 0.05 * r * k.norm(dim=-1, keepdim=True) / r.norm(dim=-1, keepdim=True)
    sink = torch.from_numpy(_sinks(c)).to(DEV).repeat_interleave(m, 1)[..., None]
    return torch.where(sink, near, active).to(torch.bfloat16)


def _cache8(c, seed, role):
    """An 8-bit cache that holds quantised rows."""
    shape = (c["b"], c["hkv"], c["lmax"])
    k, ks = _plain_quantise(_rows((*shape, D), _gen(seed, role)), c["kv"])
    v, vs = _plain_quantise(_rows((*shape, D), _gen(seed, role + 1)), c["kv"])
    return k, v, torch.stack([ks, vs], -1).contiguous()


def _dtype(c):
    return torch.float8_e4m3fn if c["kv"] == "e4m3" else torch.int8


def prepare(case, seed):
    c = dict(case)
    s = {"c": c}
    b, hkv = c["b"], c["hkv"]
    if c["op"] in ("write", "read"):
        st, n = _counts(c)
        s["start"], s["n"] = _ints(st), _ints(n)
    if c["op"] == "write":
        shape = (b, c["t"], hkv, D)
        if c["fused"]:  # columns of one projection: query heads first, then keys, then values
            qkv = _rows((b, c["t"], 4 * hkv, D), _gen(seed, 1))
            s["k_new"], s["v_new"] = qkv[:, :, 2 * hkv:3 * hkv], qkv[:, :, 3 * hkv:]
        else:
            s["k_new"], s["v_new"] = _rows(shape, _gen(seed, 1)), _rows(shape, _gen(seed, 2))
        s["k"] = torch.zeros((b, hkv, c["lmax"], D), device=DEV).to(_dtype(c))
        s["v"] = torch.zeros((b, hkv, c["lmax"], D), device=DEV).to(_dtype(c))
        s["scales"] = torch.zeros((b, hkv, c["lmax"], 2), device=DEV)
        s["k0"] = torch.zeros((b, hkv, D), device=DEV, dtype=torch.bfloat16)
        s["v0"] = torch.zeros((b, hkv, D), device=DEV, dtype=torch.bfloat16)
    elif c["op"] == "read":
        s["k"], s["v"], s["scales"] = _cache8(c, seed, 1)
        s["k_out"] = torch.zeros((b, hkv, c["t"], D), device=DEV, dtype=torch.bfloat16)
        s["v_out"] = torch.zeros((b, hkv, c["t"], D), device=DEV, dtype=torch.bfloat16)
    elif c["op"] == "append":
        s["k"] = torch.zeros((b, hkv, c["lmax"], D), device=DEV).to(_dtype(c))
        s["v"] = torch.zeros((b, hkv, c["lmax"], D), device=DEV).to(_dtype(c))
        s["scales"] = torch.zeros((b, hkv, c["lmax"], 2), device=DEV)
        s["k0"], s["v0"] = _rows((b, hkv, D), _gen(seed, 1)), _rows((b, hkv, D), _gen(seed, 2))
        s["lens"] = _ints([n - 1 for n in _lens(c)])
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["cos"], s["sin"] = _tables(c["lmax"])
        s["k_new"], s["v_new"] = _rows((b, hkv, D), _gen(seed, 3)), _rows((b, hkv, D), _gen(seed, 4))
        # the query before its rotation: the planted one rotated back
        first = s["lens"].long() == 0
        k_first = torch.where(first[:, None, None], s["k_new"], s["k0"])  # at slot 0 the new key is the position-0 key
        q = _queries(c, k_first, _gen(seed, 5)).double()
        at = s["lens"].long()
        s["q"] = _rotate(q, s["cos"][at].double(), -s["sin"][at].double()).to(torch.bfloat16)
    else:
        if c["kv"] in ("e4m3", "int8"):
            s["k"], s["v"], s["scales"] = _cache8(c, seed, 1)
        elif c["kv"] == "bf16":
            s["k"], s["v"] = (_rows((b, hkv, c["lmax"], D), _gen(seed, r)) for r in (1, 2))
            s["scales"] = None
        if c["kv"] != "none":
            s["lens"] = _ints(_lens(c))
        if c["op"] == "prefix":
            s["k_prefix"], s["v_prefix"] = (_rows((hkv, c["lp"], D), _gen(seed, r)) for r in (3, 4))
            s["k0"] = s["k_prefix"][None, :, 0].expand(b, -1, -1).contiguous()
            s["v0"] = s["v_prefix"][None, :, 0].expand(b, -1, -1).contiguous()
        else:
            s["k0"], s["v0"] = _rows((b, hkv, D), _gen(seed, 5)), _rows((b, hkv, D), _gen(seed, 6))
        s["q"] = _queries(c, s["k0"], _gen(seed, 7))
        s["mask"] = torch.from_numpy(_sinks(c)).to(DEV).to(torch.uint8).reshape(-1)
        units = torch.nonzero(s["mask"] == 0).reshape(-1).to(torch.int32)
        s["active"] = torch.zeros(1 + b * hkv, dtype=torch.int32, device=DEV)
        s["active"][0] = units.numel()
        s["active"][1:1 + units.numel()] = units
        if own:
            from kv_cache_routing_sr_b200 import native, shared_prefix
            if c["op"] == "decode":
                s["workspace"] = native.Workspace(b, hkv * c["m"], hkv, c["lmax"])
                s["out"] = torch.zeros_like(s["q"])
            elif c["kv"] == "none":
                s["workspace"] = native.PrefixWorkspace(b, hkv * c["m"], hkv, c["lp"])
                s["out"] = torch.zeros_like(s["q"])
                s["lse"] = torch.zeros(s["q"].shape[:2], device=DEV)
            else:
                s["decoder"] = shared_prefix.SharedPrefixDecoder(b, hkv * c["m"], hkv, c["lp"], c["lmax"])
    return s


# ---- the operators' plain forms --------------------------------------------------------

def _plain_quantise(x, kv):
    """Codes and scales of rows, in 32 bits. e4m3: the power of two that brings the row's largest magnitude into
    (224, 448]. int8: largest magnitude / 127. Rounded to nearest, ties to even."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True).clamp_min(FLOOR)
    if kv == "e4m3":
        f, e = torch.frexp(top)  # top = f 2^e, f in [1/2, 1); 448 = 7/8 2^9
        scale = torch.ldexp(torch.ones_like(top), e - 9 + (f > 0.875).to(e.dtype))
        return (x / scale).to(torch.float8_e4m3fn), scale[..., 0]
    return torch.round(127 * x / top).to(torch.int8), (top / 127)[..., 0]


def _rotate(x, cos, sin):
    """Rotate-half rotary embedding of [b, h, 128] with [b, 64] tables, in the type it is given."""
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    cos, sin = cos[:, None], sin[:, None]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)


def _plain_round_bf16(x):
    """64-bit values to the nearest bf16, ties to even, in one rounding."""
    f, e = torch.frexp(x)
    return torch.ldexp(torch.round(f * 256), e - 8).to(torch.bfloat16)


def _plain_write(s):
    c = s["c"]
    steps = torch.arange(c["t"], device=DEV)
    keep = steps[None, :] < s["n"][:, None]
    bi, ti = torch.nonzero(keep, as_tuple=True)
    slot = s["start"].long()[bi] + ti
    k, ks = _plain_quantise(s["k_new"], c["kv"])
    v, vs = _plain_quantise(s["v_new"], c["kv"])
    sc = torch.stack([ks, vs], -1)
    # index in the codes' bytes
    s["k"].view(torch.uint8)[bi, :, slot] = k.view(torch.uint8)[bi, ti]
    s["v"].view(torch.uint8)[bi, :, slot] = v.view(torch.uint8)[bi, ti]
    s["scales"][bi, :, slot] = sc[bi, ti]
    first = ((s["start"] == 0) & (s["n"] > 0))[:, None, None]
    s["k0"].copy_(torch.where(first, s["k_new"][:, 0], s["k0"]))
    s["v0"].copy_(torch.where(first, s["v_new"][:, 0], s["v0"]))
    return s["k"], s["v"], s["scales"], s["k0"], s["v0"]


def _plain_read(s):
    c = s["c"]
    steps = torch.arange(c["t"], device=DEV)
    keep = (steps[None, :] < s["n"][:, None])[:, None, :, None]
    at = (s["start"].long()[:, None] + steps[None, :]).clamp_max(c["lmax"] - 1)
    bi = torch.arange(c["b"], device=DEV)[:, None]
    sc = s["scales"][bi, :, at]  # [b, t, hkv, 2]
    k = s["k"].view(torch.uint8)[bi, :, at].view(_dtype(c)).float() * sc[..., :1]
    v = s["v"].view(torch.uint8)[bi, :, at].view(_dtype(c)).float() * sc[..., 1:]
    s["k_out"].copy_(torch.where(keep, k.transpose(1, 2).to(torch.bfloat16), s["k_out"]))
    s["v_out"].copy_(torch.where(keep, v.transpose(1, 2).to(torch.bfloat16), s["v_out"]))
    return s["k_out"], s["v_out"]


def _plain_route(q, k0, m):
    """1 where every head of the group has a cosine of at least TAU to the position-0 key."""
    q, k = q.float(), k0.float().repeat_interleave(m, 1)
    cos = (q * k).sum(-1) / (q.norm(dim=-1) * k.norm(dim=-1))
    return (cos.unflatten(1, (-1, m)).amin(-1) >= TAU).to(torch.uint8)


def _plain_append(s):
    c = s["c"]
    at = s["lens"].long()
    cos, sin = s["cos"][at].double(), s["sin"][at].double()
    q = _plain_round_bf16(_rotate(s["q"].double(), cos, sin))
    k = _plain_round_bf16(_rotate(s["k_new"].double(), cos, sin))
    kc, ks = _plain_quantise(k, c["kv"])
    vc, vs = _plain_quantise(s["v_new"], c["kv"])
    bi = torch.arange(c["b"], device=DEV)
    s["k"].view(torch.uint8)[bi, :, at] = kc.view(torch.uint8)
    s["v"].view(torch.uint8)[bi, :, at] = vc.view(torch.uint8)
    s["scales"][bi, :, at] = torch.stack([ks, vs], -1)
    first = (at == 0)[:, None, None]
    s["k0"].copy_(torch.where(first, k, s["k0"]))
    s["v0"].copy_(torch.where(first, s["v_new"], s["v0"]))
    mask = _plain_route(q, s["k0"], c["m"])
    s["lens_out"].copy_(s["lens"] + 1)
    return q, s["k"], s["v"], s["scales"], s["k0"], s["v0"], mask.reshape(-1), s["lens_out"]


def _plain_logits(s, q):
    """Scaled logits [b, hkv, m, lmax] over each sequence's own cache, -inf behind its length, and its values."""
    c = s["c"]
    k, v = s["k"].float(), s["v"].float()
    if s["scales"] is not None:
        k, v = k * s["scales"][..., :1], v * s["scales"][..., 1:]
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    seen = torch.arange(c["lmax"], device=DEV)[None, :] < s["lens"][:, None]
    return x.masked_fill(~seen[:, None, None, :], -math.inf), v


def _plain_finish(s, out, mask):
    c = s["c"]
    sink = mask.reshape(c["b"], c["hkv"]).bool().repeat_interleave(c["m"], 1)[..., None]
    return torch.where(sink, s["v0"].repeat_interleave(c["m"], 1), out.flatten(1, 2).to(torch.bfloat16))


def _plain_decode(s):
    c = s["c"]
    q = s["q"].float().unflatten(1, (c["hkv"], c["m"]))
    x, v = _plain_logits(s, q)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return _plain_finish(s, torch.matmul(e, v) / e.sum(-1, keepdim=True), s["mask"])


def _plain_prefix(s):
    c = s["c"]
    b, hkv, m = c["b"], c["hkv"], c["m"]
    q = s["q"].float().unflatten(1, (hkv, m))
    rows = q.transpose(0, 1).reshape(hkv, b * m, D)
    x = torch.matmul(rows, s["k_prefix"].float().transpose(-1, -2)) / math.sqrt(D)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total, out = e.sum(-1, keepdim=True), torch.matmul(e, s["v_prefix"].float())
    top, total, out = (t.unflatten(1, (b, m)).transpose(0, 1) for t in (top, total, out))
    if c["kv"] == "none":
        sink = s["mask"].reshape(b, hkv).bool().repeat_interleave(m, 1)
        lse = (top + torch.log(total)).flatten(1)
        return _plain_finish(s, out / total, s["mask"]), lse.masked_fill(sink, math.nan)
    y, v = _plain_logits(s, q)
    both = torch.maximum(top, y.amax(-1, keepdim=True))
    f, keep = torch.exp(y - both), torch.exp(top - both)
    out = (out * keep + torch.matmul(f, v)) / (total * keep + f.sum(-1, keepdim=True))
    mask = _plain_route(s["q"], s["k0"], m)
    return _plain_finish(s, out, mask), mask.reshape(-1)


# ---- one pass --------------------------------------------------------------------------

def _own(s):
    from kv_cache_routing_sr_b200 import native
    c = s["c"]
    if c["op"] == "write":
        native.kv_append_quant(s["k_new"], s["v_new"], s["start"], s["n"], s["k"], s["v"], s["scales"], s["k0"], s["v0"])
        return s["k"], s["v"], s["scales"], s["k0"], s["v0"]
    if c["op"] == "read":
        return native.kv_dequant(s["k"], s["v"], s["scales"], s["start"], s["n"], s["k_out"], s["v_out"])
    if c["op"] == "append":
        q, mask, _ = native.rope_append_route_kv(s["q"], s["k_new"], s["v_new"], s["cos"], s["sin"], s["lens"], s["k"],
                                                 s["v"], s["scales"], s["k0"], s["v0"], TAU, seq_lens_out=s["lens_out"])
        return q, s["k"], s["v"], s["scales"], s["k0"], s["v0"], mask, s["lens_out"]
    if c["op"] == "decode":
        return native.decode_attention_quant(s["q"], s["k"], s["v"], s["scales"], s["v0"], s["lens"], s["active"],
                                             out=s["out"], workspace=s["workspace"])
    if c["kv"] == "none":
        return native.prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], c["lp"], s["v0"], s["mask"], out=s["out"],
                                       lse=s["lse"], workspace=s["workspace"]), s["lse"]
    dec = s["decoder"]
    out = dec.step(s["q"], s["k_prefix"], s["v_prefix"], c["lp"], s["k"], s["v"], s["k0"], s["v0"], s["lens"], TAU,
                   kv_scales=s["scales"])
    return out, dec.route_mask


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "append": _plain_append, "decode": _plain_decode,
            "prefix": _plain_prefix}[state["c"]["op"]](state)


# ---- definitions in 64 bits ------------------------------------------------------------

def _exact_codes(x, kv):
    """(codes as the numbers they are, scales) of 64-bit rows, from the definition: the nearest number of the type's
    grid to x / scale, the even one of two."""
    top = torch.clamp(x.abs().amax(-1), min=FLOOR)
    if kv == "int8":
        return torch.round(127 * x / top[..., None]), top / 127
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
    scale = torch.where(top / scale > 448, scale * 2, scale)  # log2 may round across a power of two
    scale = torch.where(top / scale <= 224, scale / 2, scale)
    y = x / scale[..., None]
    power = torch.clamp(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))), min=-6)
    step = torch.exp2(power - 3)
    return torch.round(y / step) * step, scale


def _nearest_bf16(x):
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(1e-30))) - 7)
    return torch.round(x / step) * step


def _exact_softmax(q, k, v):
    """(attention of rows q over k and v, log of the sum of exponentials), 64 bits."""
    x = q @ k.T / math.sqrt(D)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    return (e @ v) / total, (top + torch.log(total))[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    b, hkv = c["b"], c["hkv"]
    if c["op"] == "write":
        start, n = _counts(c)
        k, v, sc = (torch.zeros(s[name].shape, dtype=torch.float64, device=DEV) for name in ("k", "v", "scales"))
        k0, v0 = s["k0"].double(), s["v0"].double()
        for i in range(b):
            for new, to, part, first in ((s["k_new"], k, 0, k0), (s["v_new"], v, 1, v0)):
                rows = new[i, :n[i]].double().transpose(0, 1)
                codes, scale = _exact_codes(rows, c["kv"])
                to[i, :, start[i]:start[i] + n[i]] = codes
                sc[i, :, start[i]:start[i] + n[i], part] = scale
                if start[i] == 0 and n[i] > 0:
                    first[i] = rows[:, 0]
        whole = c["kv"] == "int8"
        return None if whole else k, None if whole else v, sc, k0, v0
    if c["op"] == "read":
        start, n = _counts(c)
        out = [s["k_out"].double(), s["v_out"].double()]
        for i in range(b):
            rows = slice(start[i], start[i] + n[i])
            for j, name in enumerate(("k", "v")):
                out[j][i, :, :n[i]] = s[name][i, :, rows].double() * s["scales"][i, :, rows, j:j + 1].double()
        return tuple(out)
    if c["op"] == "append":
        lens = s["lens"].tolist()
        q, k_new, v_new = s["q"].double(), s["k_new"].double(), s["v_new"].double()
        k, v, sc = (torch.zeros(s[name].shape, dtype=torch.float64, device=DEV) for name in ("k", "v", "scales"))
        k0, v0 = s["k0"].double(), s["v0"].double()
        for i in range(b):
            w = torch.complex(s["cos"][lens[i]].double(), s["sin"][lens[i]].double())
            for x in (q, k_new):
                turned = torch.complex(x[i, :, :D // 2].contiguous(), x[i, :, D // 2:].contiguous()) * w
                x[i] = torch.cat([turned.real, turned.imag], -1)
            key = _nearest_bf16(k_new[i])  # the cache quantises the rotated key as bf16 holds it
            if lens[i] == 0:
                k0[i], v0[i] = key, v_new[i]
            k[i, :, lens[i]], sc[i, :, lens[i], 0] = _exact_codes(key, c["kv"])
            v[i, :, lens[i]], sc[i, :, lens[i], 1] = _exact_codes(v_new[i], c["kv"])
        whole = c["kv"] == "int8"
        return q, None if whole else k, None if whole else v, sc, k0, v0, None, None
    m = c["m"]
    lens = _lens(c) if c["kv"] != "none" else [0] * b
    sink = _sinks(c)
    out = s["v0"].double().repeat_interleave(m, 1)
    lse = torch.full(out.shape[:2], math.nan, dtype=torch.float64, device=DEV)
    for g in range(hkv):
        at = [i for i in range(b) if not sink[i][g]]
        parts = []
        if c["op"] == "prefix" and at:
            q = s["q"][at, g * m:(g + 1) * m].double().reshape(-1, D)
            o, z = _exact_softmax(q, s["k_prefix"][g].double(), s["v_prefix"][g].double())
            out[at, g * m:(g + 1) * m], lse[at, g * m:(g + 1) * m] = o.reshape(-1, m, D), z.reshape(-1, m)
        for i in at:
            if c["kv"] == "none":
                continue
            k, v = s["k"][i, g, :lens[i]].double(), s["v"][i, g, :lens[i]].double()
            if s["scales"] is not None:
                k, v = k * s["scales"][i, g, :lens[i], :1].double(), v * s["scales"][i, g, :lens[i], 1:].double()
            heads = slice(g * m, (g + 1) * m)
            o, z = _exact_softmax(s["q"][i, heads].double(), k, v)
            if c["op"] == "prefix":
                both = torch.logaddexp(lse[i, heads], z)
                o = out[i, heads] * torch.exp(lse[i, heads] - both)[:, None] + o * torch.exp(z - both)[:, None]
            out[i, heads] = o
    if c["op"] == "decode":
        return out
    return (out, lse) if c["kv"] == "none" else (out, None)
