"""Attention over a prefix that the batch shares, alone and joined with each
sequence's suffix, against 64 bits (tests/quant_ref.py).

Bars: sink heads are v0 bit for bit. Active heads are inside the elementwise bound
of the kernel's roundings: softmax weights to bf16 (half a step, 2^-8), output to
bf16 (2^-8), fp32 logits, statistics and sums."""
from __future__ import annotations

import math

import pytest
import torch

import oracle
from kv_cache_routing_sr_b200 import inputs, native, shared_prefix
from tests import quant_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TAU = 0.6


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(shape, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=gen(seed), device=DEV)).to(torch.bfloat16)


def check(q, parts_of, v0, mask, out, lse, half_out=R.HALF_BF16):
    """parts_of(b, g, heads): attention() results whose union the unit attends to."""
    B, Hq, _ = q.shape
    Hkv = v0.shape[1]
    M = Hq // Hkv
    for b in range(B):
        for g in range(Hkv):
            h = slice(g * M, (g + 1) * M)
            if mask[b][g]:
                assert torch.equal(out[b, h].float(), v0[b, g].float().expand(M, -1))
                assert lse is None or torch.isnan(lse[b, h]).all()
                continue
            o, z, a, delta = R.join(parts_of(b, g, q[b, h]))
            if torch.isinf(z).all():
                assert (out[b, h] == 0).all() and (lse is None or (lse[b, h] == -math.inf).all())
                continue
            lim = R.bound(o, a, delta, R.HALF_BF16, half_out)
            err = (out[b, h].double() - o).abs()
            assert (err <= lim).all(), f"unit {b},{g}: {float((err / lim).max())} of the bound"
            if lse is not None:
                assert ((lse[b, h].double() - z).abs() <= R.lse_bound(z, delta)).all(), f"lse of unit {b},{g}"


CASES = [
    # B, Hkv, M, prefix_len, capacity
    (1, 1, 1, 1, 1),
    (1, 8, 4, 0, 5),
    (2, 8, 4, 127, 130),
    (3, 32, 1, 577, 577),
    (5, 4, 2, 128, 128),
    (7, 3, 8, 129, 400),
    (33, 2, 4, 1000, 1001),   # 132 rows a KV head
    (40, 2, 8, 2500, 2500),   # 320 rows
    (64, 1, 8, 257, 300),     # 512 rows
    (2, 2, 8, 40000, 40000),  # long, few rows: many splits
    (5, 3, 8, 4095, 4096),    # the last length of a short prefix, and the first of a long one
    (5, 3, 8, 4096, 4096),
    (16, 5, 8, 8191, 8192),   # 128 rows a KV head
    (2, 40, 2, 4500, 4500),   # 40 items of few rows over a long prefix
    (1, 1, 1, 9000, 9001),
    (129, 3, 1, 384, 384),
    (70, 8, 8, 3001, 3001),   # 24 items of 24 tiles: a CTA's share ends one item and begins the next
    (3, 64, 1, 2100, 2100),   # 64 items of few rows, likewise
    (20, 33, 8, 700, 700),    # 160 rows a KV head: every item has more than one row tile
    (1, 700, 1, 70, 71),      # more KV heads than the plan takes at a time
    (1500, 1, 2, 65, 65),     # one KV head, twelve items
]


@pytest.mark.parametrize("B,Hkv,M,Lp,cap", CASES, ids=[f"B{c[0]}Hkv{c[1]}M{c[2]}L{c[3]}" for c in CASES])
def test_prefix_against_64_bits(B, Hkv, M, Lp, cap):
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((Hkv, cap, R.D), 3), randn((Hkv, cap, R.D), 4)
    k[:, Lp:], v[:, Lp:] = math.nan, math.nan  # behind the prefix: never used
    mask = (torch.rand(B, Hkv, generator=gen(5), device=DEV) < 0.25).to(torch.uint8)
    mask[0, 0] = 0
    ws = native.PrefixWorkspace(B, Hkv * M, Hkv, cap)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = native.prefix_attention(q, k, v, Lp, v0, mask.reshape(-1), lse=lse, workspace=ws)
    o, z = native.prefix_attention_partial(q, k, v, Lp, v0, mask.reshape(-1), workspace=ws)
    assert ws.device_error() == 0
    assert torch.equal(torch.nan_to_num(z, nan=-7.0), torch.nan_to_num(lse, nan=-7.0))
    part = lambda b, g, rows: [R.attention(rows, k[g], v[g], Lp)]  # noqa: E731
    check(q, part, v0, mask.tolist(), out, lse)
    check(q, part, v0, mask.tolist(), o, z, R.HALF_F32)


@pytest.mark.parametrize("fill", ["all", "none", "one_group", "one_row"])
def test_prefix_masks(fill):
    B, Hkv, M, Lp = 6, 4, 4, 300
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((Hkv, Lp, R.D), 3), randn((Hkv, Lp, R.D), 4)
    mask = torch.zeros(B, Hkv, dtype=torch.uint8, device=DEV)
    if fill == "all":
        mask[:] = 1
    elif fill == "one_group":
        mask[:, 2] = 255  # any value but 0 is a sink
    elif fill == "one_row":
        mask[:] = 1
        mask[5, 1] = 0
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = native.prefix_attention(q, k, v, Lp, v0, mask.reshape(-1), lse=lse)
    check(q, lambda b, g, rows: [R.attention(rows, k[g], v[g], Lp)], v0, mask.tolist(), out, lse)


@pytest.mark.parametrize("case", ["late_peak", "early_peak", "rising", "zero_q", "large_v"])
def test_prefix_extreme_logits(case):
    """Running maxima that jump late, never, or in every tile."""
    B, Hkv, M, Lp = 3, 2, 8, 1700
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((Hkv, Lp, R.D), 3, 0.2).float(), randn((Hkv, Lp, R.D), 4)
    dirn = q[0, 0].float() / q[0, 0].float().norm()
    if case == "late_peak":
        k[:, 1650] = 90 * dirn
    elif case == "early_peak":
        k[:, 3] = 90 * dirn
    elif case == "rising":
        k += torch.linspace(0, 60, Lp, device=DEV)[None, :, None] * dirn
    elif case == "zero_q":
        q.zero_()
    elif case == "large_v":
        v = (v.float() * 1e30).to(torch.bfloat16)
    k = k.to(torch.bfloat16)
    mask = torch.zeros(B * Hkv, dtype=torch.uint8, device=DEV)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = native.prefix_attention(q, k, v, Lp, v0, mask, lse=lse)
    check(q, lambda b, g, rows: [R.attention(rows, k[g], v[g], Lp)], v0, mask.view(B, Hkv).tolist(), out, lse)


@pytest.mark.parametrize("B,M,Lp", [(2, 4, 500), (40, 8, 500), (2, 4, 6000)], ids=["narrow", "wide", "wide_few_rows"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_prefix_propagates_nan(where, B, M, Lp):
    """A NaN inside the prefix reaches every active row of its KV head, and no other."""
    Hkv = 3
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((Hkv, Lp, R.D), 3), randn((Hkv, Lp, R.D), 4)
    (k if where == "k" else v)[1, 333, 5] = math.nan
    mask = torch.zeros(B, Hkv, dtype=torch.uint8, device=DEV)
    mask[0, 1] = 1
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = native.prefix_attention(q, k, v, Lp, v0, mask.reshape(-1), lse=lse).view(B, Hkv, M, R.D)
    assert torch.isfinite(out[:, [0, 2]]).all() and torch.equal(out[0, 1], v0[0, 1].expand(M, -1))
    bad = torch.isnan(out[1:, 1])
    assert bad.all() if where == "k" else (bad[..., 5].all() and not bad[..., :5].any() and not bad[..., 6:].any())


def suffix_of(kind, B, Hkv, n, seed):
    k, v = randn((B, n, Hkv, R.D), seed), randn((B, n, Hkv, R.D), seed + 1)
    if kind == "bf16":
        return k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(), None
    c = native.QuantCache(B, Hkv, n, R.E4M3 if kind == "e4m3" else R.INT8)
    z = torch.zeros(B, dtype=torch.int32, device=DEV)
    native.kv_append_quant(k, v, z, z + n, c.k, c.v, c.scales)
    return c.k, c.v, c.scales


def suffix_rows(k, v, sc, b, g, n):
    if sc is None:
        return k[b, g, :n], v[b, g, :n]
    return tuple(t[b, g, :n].double() * sc[b, g, :n, i:i + 1].double() for i, t in enumerate((k, v)))


@pytest.mark.parametrize("kind", ["bf16", *R.IDS])
@pytest.mark.parametrize("B,Hkv,M,Lp", [(2, 8, 4, 600), (9, 4, 8, 77), (5, 32, 1, 0), (40, 2, 4, 129)])
def test_shared_prefix_step(B, Hkv, M, Lp, kind):
    cap, n = max(1, Lp), 90
    lens = [1 + (31 * b) % n for b in range(B)]
    k0, v0 = randn((B, Hkv, R.D), 5), randn((B, Hkv, R.D), 6)
    q = randn((B, Hkv * M, R.D), 1)
    for b in range(B):  # some sinks
        g = b % Hkv
        q[b, g * M:(g + 1) * M] = (k0[b, g].float() + 0.05 * q[b, g * M:(g + 1) * M].float()).to(torch.bfloat16)
    kp, vp = randn((Hkv, cap, R.D), 3), randn((Hkv, cap, R.D), 4)
    ks, vs, sc = suffix_of(kind, B, Hkv, n, 7)
    dec = shared_prefix.SharedPrefixDecoder(B, Hkv * M, Hkv, cap, n)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = dec.step(q, kp, vp, Lp, ks, vs, k0, v0, sl, TAU, kv_scales=sc)
    mask = dec.route_mask.view(B, Hkv).tolist()
    assert all(mask[b][b % Hkv] for b in range(B)) and (B * Hkv <= 32 or not all(all(m) for m in mask))
    parts = lambda b, g, rows: [R.attention(rows, kp[g], vp[g], Lp),  # noqa: E731
                                R.attention(rows, *suffix_rows(ks, vs, sc, b, g, lens[b]), lens[b])]
    check(q, parts, v0, mask, out, None)
    # combine_partials on the two parts gives the same heads
    o, z = native.prefix_attention_partial(q, kp, vp, Lp, v0, dec.route_mask, workspace=dec.workspace)
    stride = (o.numel() + 3) // 4 * 4
    both_o = torch.zeros(2 * stride, device=DEV)
    both_z = torch.zeros(2 * stride, device=DEV)
    for i, (x, y) in enumerate(((o, z), (dec.o_suffix, dec.lse_suffix))):
        both_o[i * stride:i * stride + x.numel()] = x.reshape(-1)
        both_z[i * stride:i * stride + y.numel()] = y.reshape(-1)
    joined = native.combine_partials(both_o, both_z, stride, 2, B, Hkv * M)
    check(q, parts, v0, mask, joined, None)


@pytest.mark.parametrize("B,Hkv,M,cap,top", [(4, 8, 4, 9, 9), (7, 32, 1, 2, 2), (54, 32, 1, 40, 3), (60, 4, 8, 300, 300),
                                            (1, 1, 1, 1, 1)])
def test_short_bf16_suffixes_by_unit(B, Hkv, M, cap, top):
    """SPLITS_BY_UNIT against 64 bits, and against the shares of whole tiles."""
    lens = [1 + (7 * b + top - 1) % top for b in range(B)]
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((B, Hkv, cap, R.D), 3), randn((B, Hkv, cap, R.D), 4)
    mask = [[(3 * b + g) % 5 == 4 for g in range(Hkv)] for b in range(B)]
    units = [b * Hkv + g for b in range(B) for g in range(Hkv) if not mask[b][g]]
    active = torch.tensor([len(units), *units] + [-1] * (B * Hkv - len(units)), dtype=torch.int32, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = native.Workspace(B, Hkv * M, Hkv, cap)
    for b in range(B):
        k[b, :, lens[b]:], v[b, :, lens[b]:] = math.nan, math.nan
    parts = lambda b, g, rows: [R.attention(rows, k[b, g], v[b, g], lens[b])]  # noqa: E731
    for ns in (native.SPLITS_BY_UNIT, 0):
        o, z = native.decode_attention_partial(q, k, v, None, v0, sl, active, n_splits=ns, workspace=ws)
        assert ws.device_error() == 0
        check(q, parts, v0, mask, o, z, R.HALF_F32)
    o2, z2 = native.decode_attention_partial(q, k, v, None, v0, sl, active, n_splits=native.SPLITS_BY_UNIT)
    o1, z1 = native.decode_attention_partial(q, k, v, None, v0, sl, active, n_splits=native.SPLITS_BY_UNIT, workspace=ws)
    assert torch.equal(o1, o2) and torch.equal(torch.nan_to_num(z1, nan=-7.0), torch.nan_to_num(z2, nan=-7.0))


def test_join_with_an_empty_part():
    """A suffix (or prefix) without a position weighs nothing; both empty give 0."""
    B, Hkv, M, Lp = 2, 2, 4, 50
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((Hkv, Lp, R.D), 3), randn((Hkv, Lp, R.D), 4)
    mask = torch.tensor([0, 1, 0, 0], dtype=torch.uint8, device=DEV)
    o_s = torch.randn(B, Hkv * M, R.D, generator=gen(8), device=DEV)
    z_s = torch.full((B, Hkv * M), -math.inf, device=DEV)
    alone, joined = torch.zeros(B, Hkv * M, device=DEV), torch.zeros(B, Hkv * M, device=DEV)
    a = native.prefix_attention(q, k, v, Lp, v0, mask, lse=alone)
    b = native.prefix_attention(q, k, v, Lp, v0, mask, lse=joined, o_suffix=o_s, lse_suffix=z_s)
    assert torch.equal(a, b)
    keep = ~torch.isnan(alone)
    assert torch.equal(torch.isnan(joined), ~keep) and torch.allclose(alone[keep], joined[keep], rtol=1e-6)
    both = native.prefix_attention(q, k, v, 0, v0, mask, lse=joined, o_suffix=o_s, lse_suffix=z_s)
    assert (joined[keep] == -math.inf).all() and (both[keep] == 0).all()
    z_s.fill_(1.5)
    one = native.prefix_attention(q, k, v, 0, v0, mask, lse=joined, o_suffix=o_s, lse_suffix=z_s)
    assert torch.equal(one[keep], o_s.to(torch.bfloat16)[keep]) and (joined[keep] == 1.5).all()


def test_prefix_repeats_in_a_graph_and_on_a_side_stream():
    B, Hkv, M, Lp, n = 9, 4, 8, 3000, 64
    q, k0, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2), randn((B, Hkv, R.D), 3)
    kp, vp = randn((Hkv, Lp, R.D), 4), randn((Hkv, Lp, R.D), 5)
    ks, vs, sc = suffix_of("e4m3", B, Hkv, n, 6)
    sl = torch.full((B,), n, dtype=torch.int32, device=DEV)
    args = (q, kp, vp, Lp, ks, vs, k0, v0, sl, TAU, sc)
    dec, other = (shared_prefix.SharedPrefixDecoder(B, Hkv * M, Hkv, Lp, n) for _ in range(2))
    first = dec.step(*args).clone()
    for _ in range(5):
        assert torch.equal(dec.step(*args), first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.step(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            o2 = other.step(*args)
    dec.out.zero_()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dec.out, first) and torch.equal(o2, first)
    # new values in the bound tensors: the replay reads them
    q.copy_(randn(q.shape, 9))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dec.out, other.step(*args))


@pytest.mark.parametrize("kind", ["bf16", *R.IDS])
def test_generation_behind_a_shared_prefix(kind):
    """An 8-bit context is read back as the shared bf16 prefix; every sequence then
    appends and attends, token by token, from an empty suffix."""
    B, Hkv, M, Lp, n = 3, 4, 4, 200, 6
    Hq = Hkv * M
    src = native.QuantCache(1, Hkv, Lp, R.E4M3)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    native.kv_append_quant(randn((1, Lp, Hkv, R.D), 1), randn((1, Lp, Hkv, R.D), 2), z, z + Lp, src.k, src.v, src.scales)
    kp, vp = (torch.zeros(1, Hkv, Lp, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    native.kv_dequant(src.k, src.v, src.scales, z, z + Lp, kp, vp)
    kp, vp = kp[0], vp[0]
    k0, v0 = (x[None, :, 0].expand(B, -1, -1).contiguous() for x in (kp, vp))
    keep0 = k0.clone()
    if kind == "bf16":
        kc, vc, sc = (torch.zeros(B, Hkv, n, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2)), None, None
        kc, vc = kc
    else:
        c = native.QuantCache(B, Hkv, n, R.E4M3 if kind == "e4m3" else R.INT8)
        kc, vc, sc = c.k, c.v, c.scales
    seq = torch.zeros(B, dtype=torch.int32, device=DEV)
    cs, sn = inputs.rope_tables(Lp + n, device=DEV)
    dec = shared_prefix.SharedPrefixDecoder(B, Hq, Hkv, Lp, n)
    dummy = torch.zeros(B, Hkv, n, R.D, dtype=torch.bfloat16)
    for step in range(n):
        q, kn, vn = inputs.make_projections(B, Hq, Hkv, seed=60 + step, device=DEV)
        out = dec.append_step(q, kn, vn, cs, sn, kp, vp, Lp, kc, vc, k0, v0, seq, TAU, kv_scales=sc)
        assert seq.tolist() == [step + 1] * B and torch.equal(k0, keep0)
        ref = oracle.load().rope_append(q, kn, vn, cs[Lp:].contiguous(), sn[Lp:].contiguous(),
                                        torch.full((B,), step, dtype=torch.int32), dummy, dummy, k0, v0)
        assert torch.equal(dec.q.cpu().view(torch.int16), ref[1].view(torch.int16))
        check(dec.q, lambda b, g, rows: [R.attention(rows, kp[g], vp[g], Lp),
                                         R.attention(rows, *suffix_rows(kc, vc, sc, b, g, step + 1), step + 1)],
              v0, dec.route_mask.view(B, Hkv).tolist(), out, None)
        if kind == "bf16":
            assert torch.equal(kc[:, :, step].cpu().view(torch.int16), ref[2][:, :, step].view(torch.int16))


@pytest.mark.parametrize("B,Hkv,M,Lp", [(1, 1, 8, 40000), (16, 4, 8, 9000), (70, 8, 8, 3000), (3, 32, 1, 577)],
                         ids=["cta_a_row", "cta_four_rows", "warp_four_rows", "narrow"])
def test_join_of_parts_that_weigh_nothing_beside_a_later_one(B, Hkv, M, Lp):
    """Every eighth of the prefix in turn lies some 140 nats above the rest for every
    head, so that exactly the partials of the other eighths weigh 0 in fp32. A row has
    160, 74 and 7 or 8 partials in the three forms of the join, which takes them in
    groups of 256, 64 and 8, half a group at a time."""
    d = torch.randn(R.D, generator=gen(9), device=DEV)
    d = d / d.norm()
    q = (randn((B, Hkv * M, R.D), 1).float() + 40 * d).to(torch.bfloat16)
    v0, base, v = randn((B, Hkv, R.D), 2), randn((Hkv, Lp, R.D), 3).float(), randn((Hkv, Lp, R.D), 4)
    mask = torch.zeros(B, Hkv, dtype=torch.uint8, device=DEV)
    mask[0, 0] = B * Hkv > 1
    ws = native.PrefixWorkspace(B, Hkv * M, Hkv, Lp)
    for part in range(8):
        k = base.clone()
        k[:, part * Lp // 8:(part + 1) * Lp // 8] += 40 * d
        k = k.to(torch.bfloat16)
        lse = torch.zeros(q.shape[:2], device=DEV)
        out = native.prefix_attention(q, k, v, Lp, v0, mask.reshape(-1), lse=lse, workspace=ws)
        check(q, lambda b, g, rows: [R.attention(rows, k[g], v[g], Lp)], v0, mask.tolist(), out, lse)  # noqa: B023


@pytest.mark.parametrize("B,Hkv,M,Lp", [(2, 700, 1, 40), (16, 800, 8, 64), (1, 2000, 1, 1), (3, 300, 2, 129)],
                         ids=["B2", "B16", "one_position", "three_tiles"])
def test_items_of_one_tile(B, Hkv, M, Lp):
    """Many items a CTA of one 64-position tile each: the second stream has no step in
    them. Back to back calls keep their bits."""
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((Hkv, Lp, R.D), 3), randn((Hkv, Lp, R.D), 4)
    mask = (torch.rand(B, Hkv, generator=gen(5), device=DEV) < 0.2).to(torch.uint8)
    ws = native.PrefixWorkspace(B, Hkv * M, Hkv, Lp)
    lse = torch.zeros(q.shape[:2], device=DEV)
    outs = [native.prefix_attention(q, k, v, Lp, v0, mask.reshape(-1), lse=lse, workspace=ws) for _ in range(50)]
    assert ws.device_error() == 0
    check(q, lambda b, g, rows: [R.attention(rows, k[g], v[g], Lp)], v0, mask.tolist(), outs[0], lse)
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


@pytest.mark.parametrize("kind", ["bf16", *R.IDS])
def test_one_workspace_for_suffix_and_prefix_in_turn(kind):
    """The scans of a step on one buffer that is large enough for both, several steps in
    a row, against a buffer each: the prefix's plan stays off the decode counters."""
    B, Hkv, M, Lp, n = 5, 8, 4, 900, 4000
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    kp, vp = randn((Hkv, Lp, R.D), 3), randn((Hkv, Lp, R.D), 4)
    ks, vs, sc = suffix_of(kind, B, Hkv, n, 7)
    mask = (torch.rand(B, Hkv, generator=gen(5), device=DEV) < 0.25).to(torch.uint8).reshape(-1)
    units = (mask == 0).nonzero().reshape(-1).to(torch.int32)
    active = torch.zeros(1 + B * Hkv, dtype=torch.int32, device=DEV)
    active[0], active[1:1 + len(units)] = len(units), units
    sl = torch.tensor([n - 700 * b for b in range(B)], dtype=torch.int32, device=DEV)
    need = native.workspace_bytes(B, Hkv * M, Hkv, n), native.prefix_workspace_bytes(B, Hkv * M, Hkv, Lp)
    one = native.Workspace(B, Hkv * M, Hkv, n)
    one._allocate(max(need), None)

    def step(first, second):
        if sc is None:
            o, z = native.decode_attention_partial(q, ks, vs, None, v0, sl, active, workspace=first)
        else:
            o, z = native.decode_attention_quant_partial(q, ks, vs, sc, v0, sl, active, workspace=first)
        return o, native.prefix_attention(q, kp, vp, Lp, v0, mask, o_suffix=o, lse_suffix=z, workspace=second)

    want = step(native.Workspace(B, Hkv * M, Hkv, n), native.PrefixWorkspace(B, Hkv * M, Hkv, Lp))
    for _ in range(4):
        got = step(one, one)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert one.device_error() == 0


def stream_calls():
    """Every entry point that allocates, as (call(stream=..., workspace...), workspace bytes)."""
    B, Hkv, M, n = 2, 4, 4, 700
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v, sc = suffix_of("e4m3", B, Hkv, n, 3)
    kp, vp = randn((Hkv, n, R.D), 5), randn((Hkv, n, R.D), 6)
    sl = torch.full((B,), n, dtype=torch.int32, device=DEV)
    active = torch.arange(-1, B * Hkv, dtype=torch.int32, device=DEV)
    active[0] = B * Hkv
    mask = torch.zeros(B * Hkv, dtype=torch.uint8, device=DEV)
    cs, sn = inputs.rope_tables(n + 1, device=DEV)
    kn, k0 = randn((B, Hkv, R.D), 7), randn((B, Hkv, R.D), 8)
    lens = torch.full_like(sl, n - 1)
    done = torch.zeros_like(sl)
    ws, pws = native.Workspace(B, Hkv * M, Hkv, n), native.PrefixWorkspace(B, Hkv * M, Hkv, n)
    one = lambda x: x if isinstance(x, tuple) else (x,)  # noqa: E731
    return [
        (lambda w=ws, **a: one(native.decode_attention_quant(q, k, v, sc, v0, sl, active, workspace=w, **a)), ws),
        (lambda w=ws, **a: one(native.decode_attention_quant_partial(q, k, v, sc, v0, sl, active, workspace=w, **a)), ws),
        (lambda w=pws, **a: one(native.prefix_attention(q, kp, vp, n, v0, mask, workspace=w, **a)), pws),
        (lambda w=pws, **a: one(native.prefix_attention_partial(q, kp, vp, n, v0, mask, workspace=w, **a)), pws),
        (lambda w=None, **a: one(native.rope_append_route_kv(q, kn, kn, cs, sn, lens, k, v, sc, k0, v0, TAU,
                                                             seq_lens_out=done, **a)), None),
    ]


@pytest.mark.parametrize("i", range(5), ids=["scan", "scan_partial", "prefix", "prefix_partial", "append"])
def test_outputs_allocated_for_another_stream(i):
    """The current stream still writes tensors that have just been released there: an
    output for a side stream must not lie in their memory."""
    call, _ = stream_calls()[i]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty_like(t) for t in want for _ in range(3)]
    torch.cuda._sleep(40_000_000)
    for t in late:
        t.fill_(7)
    del late, t
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("i", range(4), ids=["scan", "scan_partial", "prefix", "prefix_partial"])
def test_a_calls_own_workspace_outlives_its_kernels_on_another_stream(i):
    """A workspace that the call allocates is released when it returns; the side stream
    has not begun yet, and the current stream takes memory of the same size."""
    call, ws = stream_calls()[i]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    got = call(w=None, stream=side)
    others = [torch.full((ws.nbytes + 256,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(others) == 4


@pytest.mark.parametrize("kind", ["bf16", *R.IDS])
@pytest.mark.parametrize("B,Hkv,M,Lp", [(2, 8, 4, 600), (9, 4, 8, 77), (5, 32, 1, 0), (40, 2, 4, 129)])
def test_shared_prefix_step_routes_the_planted_sinks_and_no_others(B, Hkv, M, Lp, kind):
    """The step's mask is the planted one, with active units in every case, and active
    heads are the attention over prefix and suffix together: neither part alone."""
    cap, n = max(1, Lp), 90
    lens = [1 + (31 * b) % n for b in range(B)]
    k0, v0 = randn((B, Hkv, R.D), 5), randn((B, Hkv, R.D), 6)
    r = randn((B, Hkv, M, R.D), 1).float()
    hat = k0.float() / k0.float().norm(dim=-1, keepdim=True)
    r = r - (r * hat[:, :, None]).sum(-1, keepdim=True) * hat[:, :, None]  # cosine 0 to the position-0 key
    planted = torch.tensor([[g == b % Hkv for g in range(Hkv)] for b in range(B)], device=DEV)
    q = torch.where(planted[..., None, None], k0[:, :, None].float() + 0.05 * r, r).to(torch.bfloat16).reshape(B, Hkv * M, R.D)
    kp, vp = randn((Hkv, cap, R.D), 3), randn((Hkv, cap, R.D), 4)
    ks, vs, sc = suffix_of(kind, B, Hkv, n, 7)
    dec = shared_prefix.SharedPrefixDecoder(B, Hkv * M, Hkv, cap, n)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = dec.step(q, kp, vp, Lp, ks, vs, k0, v0, sl, TAU, kv_scales=sc)
    mask = dec.route_mask.view(B, Hkv)
    assert torch.equal(mask, planted.to(torch.uint8)) and not bool(mask.all())
    part = [lambda b, g, rows: R.attention(rows, kp[g], vp[g], Lp),
            lambda b, g, rows: R.attention(rows, *suffix_rows(ks, vs, sc, b, g, lens[b]), lens[b])]
    check(q, lambda b, g, rows: [p(b, g, rows) for p in part], v0, mask.tolist(), out, None)
    for p in part if Lp else part[:1]:
        with pytest.raises(AssertionError):
            check(q, lambda b, g, rows: [p(b, g, rows)], v0, mask.tolist(), out, None)  # noqa: B023


def spread(n, count):
    """About `count` indices over [0, n), the last among them."""
    return sorted({*range(0, n, max(1, n // count)), n - 1})


@pytest.mark.parametrize("B,Hkv,M,Lp", [(16384, 1, 8, 70), (2048, 8, 8, 300), (16384, 1, 1, 5000), (1, 16384, 1, 2),
                                        (8, 2048, 1, 130)])
def test_largest_launches(B, Hkv, M, Lp):
    """Up to the most units and 131072 rows; a spread of sequences and heads is checked."""
    q, v0 = randn((B, Hkv * M, R.D), 1), randn((B, Hkv, R.D), 2)
    k, v = randn((Hkv, Lp, R.D), 3), randn((Hkv, Lp, R.D), 4)
    mask = (torch.rand(B, Hkv, generator=gen(5), device=DEV) < 0.25).to(torch.uint8)
    ws = native.PrefixWorkspace(B, Hkv * M, Hkv, Lp)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = native.prefix_attention(q, k, v, Lp, v0, mask.reshape(-1), lse=lse, workspace=ws)
    assert ws.device_error() == 0
    at, gs = spread(B, 30), spread(Hkv, 20)
    hs = [g * M + m for g in gs for m in range(M)]
    check(q[at][:, hs], lambda b, g, rows: [R.attention(rows, k[gs[g]], v[gs[g]], Lp)], v0[at][:, gs],
          mask[at][:, gs].tolist(), out[at][:, hs], lse[at][:, hs])


def test_far_positions_of_a_prefix_over_4_gib():
    """Positions behind 2^24 and rows behind byte offset 2^32: all keys but the last three
    are zero (logit 0), and so are all values."""
    Hkv, M, B, n = 2, 4, 3, (1 << 24) + 5
    k, v = (torch.zeros(Hkv, n, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    k[:, -3:], v[:, -3:] = randn((Hkv, 3, R.D), 1), randn((Hkv, 3, R.D), 2)
    q = (4 * k[:, -2].float()[None, :, None] + 0.1 * randn((B, Hkv, M, R.D), 3).float()).to(torch.bfloat16)
    q, v0 = q.reshape(B, Hkv * M, R.D), randn((B, Hkv, R.D), 5)
    lse = torch.zeros(B, Hkv * M, device=DEV)
    out = native.prefix_attention(q, k, v, n, v0, torch.zeros(B * Hkv, dtype=torch.uint8, device=DEV), lse=lse)
    for g in range(Hkv):
        h = slice(g * M, (g + 1) * M)
        kd, vd, rows = k[g, -3:].double(), v[g, -3:].double(), q[:, h].double().reshape(-1, R.D)
        e = torch.exp(rows @ kd.T / math.sqrt(R.D))
        tot = e.sum(-1, keepdim=True) + (n - 3)
        o, a = e @ vd / tot, e @ vd.abs() / tot
        delta = 130 * R.HALF_F32 * (rows.abs() @ kd.abs().T / math.sqrt(R.D)).amax(-1)
        # the sum of 2^24 ones in fp32: a tile's 128 in two chains, a CTA's tiles and the CTAs' partials in a row add
        # at most 2^11 of them one after another
        lim = R.bound(o, a, delta, R.HALF_BF16, R.HALF_BF16) + 2.0 ** -12 * a
        err = (out[:, h].double().reshape(-1, R.D) - o).abs()
        assert bool((err <= lim).all()), float((err / lim).max())
        z = torch.log(tot[:, 0])
        assert ((lse[:, h].double().reshape(-1) - z).abs() <= R.lse_bound(z, delta) + 2.0 ** -12).all()
