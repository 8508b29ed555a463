"""The 8-bit KV cache on the GPU: bulk writes, reads, the single-token append and
the routed scan, against their definitions in 64 bits (tests/quant_ref.py) and the
oracle's rotation.

Bars. Codes and scales are bit-exact. Rows read back are the rounding of code *
scale. The append's query, position-0 rows, mask and lengths are bit-exact with
the oracle and sr_route. The scan is inside the elementwise bound of its own
roundings: softmax weights to fp16 (half a step, 2^-11), output to bf16 (2^-8),
fp32 logits; a weight below 2^-39 of the largest may vanish (fp16's smallest step
2^-24 under the scaling by 2^14, half of it lost)."""
from __future__ import annotations

import math

import pytest
import torch

import oracle
from kv_cache_routing_sr_b200 import inputs, native
from tests import gpu_helpers as H
from tests import quant_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TAU = 0.6
both = pytest.mark.parametrize("dtype", R.DTYPES, ids=R.IDS)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows(shape, seed):
    """bf16 rows over many magnitudes, with ties, zeros and a row of zeros among them."""
    x = torch.randn(shape, generator=gen(seed), device=DEV)
    x = x * torch.exp2(torch.randint(-12, 13, (*shape[:-1], 1), generator=gen(seed + 1), device=DEV).float())
    x = x.to(torch.bfloat16)
    flat = x.view(-1, R.D)
    n = flat.shape[0]
    flat[0] = 0
    if n > 1:  # ties of both formats: top and its halves, odd multiples
        flat[1] = torch.tensor([127.0, 63.5, 0.5, 1.5, -2.5, -63.5, 254.0 / 2, 17.0] * 16, device=DEV).to(torch.bfloat16)
    if n > 2:
        flat[2] = torch.tensor([3.0, 1.5, 0.75, -1.5, 2.0, 1.0, -0.5, 0.25] * 16, device=DEV).to(torch.bfloat16)
    if n > 3:
        flat[3] = torch.tensor([448.0, 17.0, 19.0, -21.0, 2.0 ** -9, 3 * 2.0 ** -10, 2.0 ** -10, 0.0] * 16,
                               device=DEV).to(torch.bfloat16)
    if n > 4:
        flat[4] = 3e38
    if n > 5:
        flat[5] = 1e-38
    return x


def assert_rows(codes, scales, x, dtype, what):
    want, ws = R.quantise(x, dtype)
    assert torch.equal(torch.isnan(scales), torch.isnan(ws)), what
    ok = ~torch.isnan(ws)
    assert torch.equal(scales[ok], ws[ok]), f"{what}: scales differ"
    got = codes.double()
    if not torch.equal(got, want):
        bad = (got != want).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {bad.shape[0]} codes differ, first at {i}: {got[i]} for {want[i]}, "
                             f"x {x[i].item()}, scale {scales[i[:-1]].item()}")


def sentinel_cache(B, Hkv, Lmax, dtype):
    c = native.QuantCache(B, Hkv, Lmax, dtype)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x55)
    c.scales.fill_(-7.0)
    return c


WRITES = [
    # B, Hkv, T, Lmax, starts, counts
    (1, 1, 1, 1, [0], [1]),
    (1, 8, 5, 9, [0], [5]),
    (2, 5, 7, 33, [0, 26], [7, 7]),
    (3, 4, 64, 101, [37, 0, 11], [64, 0, 1]),
    (4, 32, 33, 64, [31, 0, 1, 0], [33, 2, 32, 33]),
]


@both
@pytest.mark.parametrize("fused", [False, True], ids=["own", "view"])
@pytest.mark.parametrize("B,Hkv,T,Lmax,start,count", WRITES, ids=[f"B{w[0]}T{w[2]}" for w in WRITES])
def test_append_quant_writes_exactly_its_rows(B, Hkv, T, Lmax, start, count, fused, dtype):
    if fused:
        p = rows((B, T, 3 * Hkv, R.D), 5)
        k, v = p[:, :, Hkv:2 * Hkv], p[:, :, 2 * Hkv:]
    else:
        k, v = rows((B, T, Hkv, R.D), 5), rows((B, T, Hkv, R.D), 6)
    c = sentinel_cache(B, Hkv, Lmax, dtype)
    k0 = torch.full((B, Hkv, R.D), 9.0, device=DEV, dtype=torch.bfloat16)
    v0 = k0.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    st, n = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (start, count))
    got = native.kv_append_quant(k, v, st, n, c.k, c.v, c.scales, k0, v0, device_error=err)
    assert got[0] is c.k and int(err) == 0
    seen = torch.zeros((B, Hkv, Lmax), dtype=torch.bool, device=DEV)
    for b in range(B):
        s, e = start[b], start[b] + count[b]
        seen[b, :, s:e] = True
        for new, cache, part in ((k, c.k, 0), (v, c.v, 1)):
            x = new[b, :count[b]].transpose(0, 1)
            assert_rows(cache[b, :, s:e], c.scales[b, :, s:e, part], x, dtype, f"sequence {b}")
        first = start[b] == 0 and count[b] > 0
        assert torch.equal(k0[b], k[b, 0] if first else torch.full_like(k0[b], 9.0))
        assert torch.equal(v0[b], v[b, 0] if first else torch.full_like(v0[b], 9.0))
    for t in (c.k, c.v):
        assert (t.view(torch.uint8)[~seen] == 0x55).all(), "rows behind the chunk changed"
    assert (c.scales[~seen] == -7.0).all()


@both
def test_append_quant_covers_every_bf16_ratio(dtype):
    """Every bf16 significand as the row's largest magnitude against every one as
    an element, over the exponents that reach a code: all ties, both signs."""
    tops = torch.arange(128, 256, device=DEV).double() / 128
    elems = torch.arange(128, 256, device=DEV).double() / 128
    x = torch.zeros(128, 16, 128, device=DEV, dtype=torch.float64)
    for e in range(16):
        x[:, e] = elems * 2.0 ** -e * (1 - 2 * (e % 2))
    x = torch.where(x.abs() > tops[:, None, None], torch.zeros_like(x), x)
    x[:, :, 0] = tops[:, None]
    x = x.to(torch.bfloat16).reshape(1, 2048, 1, R.D)
    c = native.QuantCache(1, 1, 2048, dtype)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    native.kv_append_quant(x, -x, z, z + 2048, c.k, c.v, c.scales)
    assert_rows(c.k[0, 0], c.scales[0, 0, :, 0], x[0, :, 0], dtype, "keys")
    assert_rows(c.v[0, 0], c.scales[0, 0, :, 1], -x[0, :, 0], dtype, "values")


@both
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_quant_non_finite_rows(dtype, bad):
    x = rows((1, 8, 2, R.D), 3)
    y = x.clone()
    y[0, 6, 1, 77] = bad
    c = native.QuantCache(1, 2, 8, dtype)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    native.kv_append_quant(y, x, z, z + 8, c.k, c.v, c.scales)
    assert_rows(c.k[0], c.scales[0, :, :, 0], y[0].transpose(0, 1), dtype, "keys")
    assert_rows(c.v[0], c.scales[0, :, :, 1], x[0].transpose(0, 1), dtype, "values")
    k, v = (torch.zeros(1, 2, 8, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    native.kv_dequant(c.k, c.v, c.scales, z, z + 8, k, v)
    assert torch.isnan(k[0, 1, 6]).all() and torch.isfinite(v).all()
    assert torch.isnan(k).sum() == R.D


@both
def test_append_quant_reports_bad_slots_and_counts(dtype):
    B, Hkv, T, Lmax = 6, 2, 4, 10
    k, v = rows((B, T, Hkv, R.D), 1), rows((B, T, Hkv, R.D), 2)
    c = sentinel_cache(B, Hkv, Lmax, dtype)
    #        runs off the end  before 0   past    bad counts       far out
    start = torch.tensor([8, -2, 10, 1, 2, 2147483647], dtype=torch.int32, device=DEV)
    count = torch.tensor([4, 4, 1, 5, -3, 4], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    native.kv_append_quant(k, v, start, count, c.k, c.v, c.scales, device_error=err)
    assert int(err) == native.SR_DEVERR_APPEND_SLOT | native.SR_DEVERR_ROW_COUNT
    seen = torch.zeros((B, Lmax), dtype=torch.bool)
    seen[0, 8:10] = seen[1, 0:2] = seen[3, 1:5] = True
    written = (c.scales[:, 0, :, 0] != -7.0).cpu()
    assert torch.equal(written, seen)
    assert_rows(c.k[0, :, 8:], c.scales[0, :, 8:, 0], k[0, :2].transpose(0, 1), dtype, "clipped")
    assert_rows(c.k[1, :, :2], c.scales[1, :, :2, 0], k[1, 2:].transpose(0, 1), dtype, "clipped")


@both
@pytest.mark.parametrize("B,Hkv,T,Lmax,start,count", WRITES, ids=[f"B{w[0]}T{w[2]}" for w in WRITES])
def test_dequant_reads_exactly_its_rows(B, Hkv, T, Lmax, start, count, dtype):
    c = native.QuantCache(B, Hkv, Lmax, dtype)
    g = gen(4)
    for t in (c.k, c.v):
        x = torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        t.view(torch.uint8).copy_(x)  # every code, e4m3's NaN among them
    c.scales.copy_(torch.randn(c.scales.shape, generator=g, device=DEV))
    st, n = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (start, count))
    k, v = (torch.full((B, Hkv, T, R.D), 5.0, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    native.kv_dequant(c.k, c.v, c.scales, st, n, k, v, device_error=err)
    assert int(err) == 0
    for out, cache, part in ((k, c.k, 0), (v, c.v, 1)):
        want = torch.full_like(out, 5.0)
        for b in range(B):
            s, e = start[b], start[b] + count[b]
            x = cache[b, :, s:e].float() * c.scales[b, :, s:e, part:part + 1]
            want[b, :, :count[b]] = x.to(torch.bfloat16)
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


def test_dequant_of_written_e4m3_rows_is_exact_and_int8_within_half_a_step():
    x = rows((1, 40, 3, R.D), 8)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    for dtype in R.DTYPES:
        c = native.QuantCache(1, 3, 40, dtype)
        native.kv_append_quant(x, x, z, z + 40, c.k, c.v, c.scales)
        k, v = (torch.zeros(1, 3, 40, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        native.kv_dequant(c.k, c.v, c.scales, z, z + 40, k, v)
        codes, scales = R.quantise(x[0].transpose(0, 1), dtype)
        want = codes * scales[..., None].double()
        if dtype == R.E4M3:
            assert torch.equal(k[0].double(), want)
        else:
            assert ((k[0].double() - want).abs() <= (R.HALF_BF16 + R.HALF_F32) * want.abs()).all()
        assert torch.equal(k, v)


# ---- append ------------------------------------------------------------------------------

APPENDS = [
    # B, Hkv, M, Lmax, positions, sink units, offset
    (2, 8, 4, 64, [0, 37], (0, 1, 9, 12), 0),
    (3, 4, 1, 64, [63, 5, 0], (2, 5, 11), 0),
    (2, 4, 2, 41, [17, 0], (0, 7), 90),
    (3, 8, 8, 16, [0, 15, 3], (3, 8, 15, 23), 5),
    (9, 32, 1, 100, [99, 0, 1, 2, 3, 50, 60, 98, 0], tuple(range(0, 288, 7)), 0),
]


def append_case(B, Hkv, M, Lmax, positions, sinks, off, seed=3):
    """Inputs whose listed units are sinks once rotated (built by rotating the
    target back with the oracle), and the oracle's state after the step."""
    g = torch.Generator().manual_seed(seed)
    q, kn, vn = inputs.make_projections(B, Hkv * M, Hkv, seed=seed)
    cs, sn = inputs.rope_tables(Lmax + off)
    k0, v0 = (torch.randn(B, Hkv, R.D, generator=g).to(torch.bfloat16) for _ in range(2))
    seq = torch.tensor(positions, dtype=torch.int32)
    dummy = torch.zeros(B, Hkv, Lmax, R.D, dtype=torch.bfloat16)
    o = oracle.load()
    run = lambda x, s: o.rope_append(x, kn, vn, cs[off:].contiguous(), s[off:].contiguous(), seq, dummy, dummy, k0, v0)  # noqa: E731
    after = run(q, sn)
    k0_after = after[4] if off == 0 else k0
    v0_after = after[5] if off == 0 else v0
    target = q.clone()
    for u in sinks:
        b, gg = divmod(u, Hkv)
        for m in range(M):
            noise = 0.03 * torch.randn(R.D, generator=g) * k0_after[b, gg].float().norm() / 11.3
            target[b, gg * M + m] = (k0_after[b, gg].float() + noise).to(torch.bfloat16)
    back = run(target, -sn)[1]
    for u in sinks:
        b, gg = divmod(u, Hkv)
        q[b, gg * M:(gg + 1) * M] = back[b, gg * M:(gg + 1) * M]
    after = run(q, sn)
    return dict(q=q, kn=kn, vn=vn, cs=cs, sn=sn, seq=seq, k0=k0, v0=v0), after, k0_after, v0_after


@pytest.mark.parametrize("dtype", [torch.bfloat16, *R.DTYPES], ids=["bf16", *R.IDS])
@pytest.mark.parametrize("separate", [False, True], ids=["inplace", "separate"])
@pytest.mark.parametrize("B,Hkv,M,Lmax,pos,sinks,off", APPENDS, ids=[f"B{a[0]}Hkv{a[1]}M{a[2]}" for a in APPENDS])
def test_append_matches_oracle(B, Hkv, M, Lmax, pos, sinks, off, separate, dtype):
    c, after, k0_ref, v0_ref = append_case(B, Hkv, M, Lmax, pos, sinks, off)
    d = {k: v.to(DEV) for k, v in c.items()}
    quant = dtype != torch.bfloat16
    if quant:
        cache = sentinel_cache(B, Hkv, Lmax, dtype)
        kc, vc, sc = cache.k, cache.v, cache.scales
    else:
        kc, vc, sc = torch.full((B, Hkv, Lmax, R.D), 3.0, device=DEV, dtype=dtype), None, None
        vc = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.full_like(d["seq"], -1) if separate else None
    q_out, mask, active = native.rope_append_route_kv(
        d["q"], d["kn"], d["vn"], d["cs"], d["sn"], d["seq"], kc, vc, sc, d["k0"], d["v0"], TAU, pos_offset=off,
        seq_lens_out=lens, device_error=err)
    assert int(err) == 0
    bits = lambda t: t.detach().cpu().contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(q_out), bits(after[1]))
    assert torch.equal(bits(d["k0"]), bits(k0_ref)) and torch.equal(bits(d["v0"]), bits(v0_ref))
    assert torch.equal((lens if separate else d["seq"]).cpu(), c["seq"] + 1)
    if separate:
        assert torch.equal(d["seq"].cpu(), c["seq"])
    m2, a2 = native.route(q_out, d["k0"], TAU)
    H.assert_route_equal(mask.cpu(), active.cpu(), m2.cpu(), a2.cpu())
    assert all(int(mask[u]) == 1 for u in sinks) and int(mask.sum()) < B * Hkv
    seen = torch.zeros((B, Hkv, Lmax), dtype=torch.bool)
    for b in range(B):
        seen[b, :, pos[b]] = True
        k_row, v_row = after[2][b, :, pos[b]], after[3][b, :, pos[b]]
        if quant:
            assert_rows(kc[b, :, pos[b]].cpu(), sc[b, :, pos[b], 0].cpu(), k_row, dtype, f"key {b}")
            assert_rows(vc[b, :, pos[b]].cpu(), sc[b, :, pos[b], 1].cpu(), v_row, dtype, f"value {b}")
        else:
            assert torch.equal(bits(kc[b, :, pos[b]]), bits(k_row)) and torch.equal(bits(vc[b, :, pos[b]]), bits(v_row))
    if quant:
        assert (kc.view(torch.uint8).cpu()[~seen] == 0x55).all() and (vc.view(torch.uint8).cpu()[~seen] == 0x55).all()
        assert (sc.cpu()[~seen] == -7.0).all()
    else:
        assert (kc.cpu()[~seen] == 3.0).all() and (vc.cpu()[~seen] == 3.0).all()


@both
def test_append_bad_slots_leave_their_sequence_alone(dtype):
    B, Hkv, M, Lmax = 4, 2, 4, 8
    c, _, _, _ = append_case(B, Hkv, M, Lmax, [1, 2, 3, 4], (), 0)
    d = {k: v.to(DEV) for k, v in c.items()}
    d["seq"] = torch.tensor([8, -1, 3, 6], dtype=torch.int32, device=DEV)  # 6 + 3 is behind the tables
    cache = sentinel_cache(B, Hkv, Lmax, dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.zeros_like(d["seq"])
    q_out, mask, _ = native.rope_append_route_kv(
        d["q"], d["kn"], d["vn"], d["cs"], d["sn"], d["seq"], cache.k, cache.v, cache.scales, d["k0"], d["v0"], TAU,
        pos_offset=3, seq_lens_out=lens, device_error=err)
    assert int(err) == native.SR_DEVERR_APPEND_SLOT
    assert lens.tolist() == [8, -1, 4, 6]
    assert (q_out[[0, 1, 3]] == 0).all() and (q_out[2] != 0).any()
    wrote = (cache.scales[:, :, :, 0] != -7.0).nonzero().tolist()
    assert wrote == [[2, 0, 3], [2, 1, 3]]


# ---- the scan ----------------------------------------------------------------------------

def filled_cache(B, Hkv, Lmax, lens, dtype, seed, spread=2.0, poison=True):
    """A cache of random rows whose scales vary by 2^+-spread from row to row, with
    NaN codes and scales behind every length."""
    c = native.QuantCache(B, Hkv, Lmax, dtype)
    z = torch.zeros(B, dtype=torch.int32, device=DEV)
    shape = (B, Lmax, Hkv, R.D)
    k, v = (torch.randn(shape, generator=gen(seed + i), device=DEV) *
            torch.exp2(spread * (2 * torch.rand((*shape[:3], 1), generator=gen(seed + 2 + i), device=DEV) - 1))
            for i in range(2))
    native.kv_append_quant(k.to(torch.bfloat16), v.to(torch.bfloat16), z, z + Lmax, c.k, c.v, c.scales)
    if poison:
        for b in range(B):
            for t in (c.k, c.v):
                t.view(torch.uint8)[b, :, lens[b]:] = 0x7f
            c.scales[b, :, lens[b]:] = math.nan
    return c


def check_scan(q, c, v0, lens, mask, out, lse, o_f32=None):
    B, Hkv, _, _ = c.k.shape
    M = q.shape[1] // Hkv
    for b in range(B):
        for g in range(Hkv):
            h = slice(g * M, (g + 1) * M)
            if mask[b][g]:
                assert torch.equal(out[b, h], v0[b, g].expand(M, -1)) and torch.isnan(lse[b, h]).all()
                continue
            k, v = (t[b, g, :lens[b]].double() * c.scales[b, g, :lens[b], i:i + 1].double()
                    for i, t in enumerate((c.k, c.v)))
            o, z, a, delta = R.attention(q[b, h], k, v, lens[b])
            under = lens[b] * 2.0 ** -39 * float(v.abs().max())
            lim = R.bound(o, a, delta, R.HALF_F16, R.HALF_BF16, under)
            err = (out[b, h].double() - o).abs()
            assert (err <= lim).all(), f"unit {b},{g}: {float((err / lim).max())} of the bound"
            assert ((lse[b, h].double() - z).abs() <= R.lse_bound(z, delta)).all(), f"lse of unit {b},{g}"
            if o_f32 is not None:
                lim = R.bound(o, a, delta, R.HALF_F16, R.HALF_F32, under)
                assert ((o_f32[b, h].double() - o).abs() <= lim).all()


def scan(q, c, v0, lens, mask, n_splits=0, stream=None):
    """Both forms of the scan; out, lse and the partials."""
    B, Hkv, Lmax, _ = c.k.shape
    units = (mask.reshape(-1) == 0).nonzero().reshape(-1).to(torch.int32)
    active = torch.full((1 + B * Hkv,), -1, dtype=torch.int32, device=DEV)
    active[0] = units.numel()
    active[1:1 + units.numel()] = units
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = native.Workspace(B, q.shape[1], Hkv, Lmax, n_splits)
    lse = torch.zeros(q.shape[:2], device=DEV)
    torch.cuda.synchronize()
    out = native.decode_attention_quant(q, c.k, c.v, c.scales, v0, sl, active, n_splits=n_splits, workspace=ws, lse=lse,
                                        stream=stream)
    o, z = native.decode_attention_quant_partial(q, c.k, c.v, c.scales, v0, sl, active, n_splits=n_splits, workspace=ws,
                                                 stream=stream)
    torch.cuda.synchronize()
    assert ws.device_error() == 0
    assert torch.equal(torch.nan_to_num(z, nan=-7.0), torch.nan_to_num(lse, nan=-7.0))
    return out, lse, o


SCANS = [
    # B, Hkv, M, Lmax, lens, n_splits
    (1, 1, 1, 1, [1], 0),
    (1, 1, 8, 129, [129], 0),  # an odd number of scale pairs, the last one read on its own
    (1, 5, 4, 131, [131], 0),
    (3, 1, 2, 257, [2, 257, 128], 0),
    (4, 8, 4, 700, [1, 127, 700, 513], 0),
    (2, 8, 8, 3001, [3001, 1400], 0),
    (5, 8, 1, 999, [999, 1, 500, 64, 65], 3),
    (1, 8, 4, 20011, [20011], 0),
    (1, 2, 8, 4099, [4099], 37),
    (40, 2, 2, 67, [1 + (13 * i) % 67 for i in range(40)], 0),  # more than 32 units
    # short units, whose shares follow the units: fewer than the grid's CTAs, more, many
    (4, 8, 4, 9, [9, 1, 3, 9], 0),
    (1, 32, 1, 255, [255], 0),
    (7, 32, 1, 2, [2, 1, 2, 2, 1, 1, 2], 0),
    (54, 32, 1, 2, [1 + i % 2 for i in range(54)], 0),
    (60, 5, 8, 3, [1 + i % 3 for i in range(60)], 0),
    (64, 8, 2, 2000, [2000] + [1 + i % 7 for i in range(63)], 0),  # one long sequence among short ones
    (3, 8, 8, 300, [300, 220, 247], 0),  # an average of just less than a whole share
]


@both
@pytest.mark.parametrize("B,Hkv,M,Lmax,lens,ns", SCANS, ids=[f"B{s[0]}Hkv{s[1]}M{s[2]}L{s[3]}s{s[5]}" for s in SCANS])
def test_scan_against_64_bits(B, Hkv, M, Lmax, lens, ns, dtype):
    c = filled_cache(B, Hkv, Lmax, lens, dtype, 11)
    q = torch.randn(B, Hkv * M, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    v0 = torch.randn(B, Hkv, R.D, generator=gen(2), device=DEV).to(torch.bfloat16)
    mask = torch.rand(B, Hkv, generator=gen(3), device=DEV) < 0.3
    mask[0, 0] = False
    out, lse, o = scan(q, c, v0, lens, mask, ns)
    check_scan(q, c, v0, lens, mask.tolist(), out, lse, o)


@both
@pytest.mark.parametrize("all_sinks", [True, False])
def test_scan_of_all_sinks_and_none(all_sinks, dtype):
    c = filled_cache(2, 4, 50, [50, 9], dtype, 5)
    q = torch.randn(2, 16, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    v0 = torch.randn(2, 4, R.D, generator=gen(2), device=DEV).to(torch.bfloat16)
    mask = torch.full((2, 4), all_sinks, device=DEV)
    out, lse, o = scan(q, c, v0, [50, 9], mask)
    check_scan(q, c, v0, [50, 9], mask.tolist(), out, lse, o)


@both
@pytest.mark.parametrize("case", ["scales", "tiny_scales", "zero_scales", "huge_q", "tiny_q", "zero_q", "one_hot", "sink_row"])
def test_scan_extreme_values(case, dtype):
    B, Hkv, M, Lmax = 1, 2, 4, 400
    lens = [387]
    c = filled_cache(B, Hkv, Lmax, lens, dtype, 21)
    q = torch.randn(B, Hkv * M, R.D, generator=gen(1), device=DEV)
    n = lens[0]
    if case == "scales":  # value scales over 2^60, in rising and falling order
        e = torch.linspace(-40, 20, n, device=DEV)
        c.scales[0, 0, :n, 1] = torch.exp2(e)
        c.scales[0, 1, :n, 1] = torch.exp2(e.flip(0))
    elif case == "tiny_scales":
        c.scales[0, :, :n, 1] = 2.0 ** -106
    elif case == "zero_scales":
        c.scales[0, :, :n, 1] = 0.0
        c.scales[0, 1, 5, 1] = 1.0
    elif case == "huge_q":
        q *= 2.0 ** 100
        c.scales[0, :, :n, 0] *= 2.0 ** -100
    elif case == "tiny_q":
        q *= 2.0 ** -90
        c.scales[0, :, :n, 0] *= 2.0 ** 90
    elif case == "zero_q":
        q.zero_()
    elif case == "one_hot":  # one element carries the row: the others are far below it
        q *= 2.0 ** -12
        q[..., 5] = 3.0
    elif case == "sink_row":  # one position takes nearly all the weight, late in the scan
        c.scales[0, :, 380, 0] *= 60.0
    q = q.to(torch.bfloat16)
    v0 = torch.zeros(B, Hkv, R.D, device=DEV, dtype=torch.bfloat16)
    mask = torch.zeros(B, Hkv, dtype=torch.bool, device=DEV)
    out, lse, o = scan(q, c, v0, lens, mask, 2)
    check_scan(q, c, v0, lens, mask.tolist(), out, lse, o)


@both
def test_scan_propagates_a_stored_nan_row(dtype):
    c = filled_cache(1, 2, 64, [64], dtype, 2)
    c.scales[0, 1, 40] = math.nan
    q = torch.randn(1, 8, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    v0 = torch.zeros(1, 2, R.D, device=DEV, dtype=torch.bfloat16)
    out, lse, _ = scan(q, c, v0, [64], torch.zeros(1, 2, dtype=torch.bool, device=DEV))
    assert torch.isfinite(out[0, :4]).all() and torch.isnan(out[0, 4:]).all()


@both
def test_scan_is_deterministic_and_repeats_in_a_graph(dtype):
    B, Hkv, M, Lmax = 2, 4, 4, 5003
    lens = [5003, 2600]
    c = filled_cache(B, Hkv, Lmax, lens, dtype, 9)
    q = torch.randn(B, Hkv * M, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    k0 = torch.randn(B, Hkv, R.D, generator=gen(4), device=DEV).to(torch.bfloat16)
    v0 = torch.randn(B, Hkv, R.D, generator=gen(2), device=DEV).to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    dec = native.QuantDecoder(B, Hkv * M, Hkv, Lmax)
    first = dec.step(q, c, k0, v0, sl, TAU).clone()
    for _ in range(5):
        assert torch.equal(dec.step(q, c, k0, v0, sl, TAU), first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.step(q, c, k0, v0, sl, TAU)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = native.QuantDecoder(B, Hkv * M, Hkv, Lmax)
    with torch.cuda.stream(side):  # another decoder's calls while the graph replays
        for _ in range(5):
            o2 = other.step(q, c, k0, v0, sl, TAU)
    dec.out.zero_()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dec.out, first) and torch.equal(o2, first)


@both
def test_scan_reports_bad_lengths_and_lists(dtype):
    c = filled_cache(2, 2, 30, [30, 30], dtype, 9, poison=False)
    q = torch.randn(2, 4, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    v0 = torch.zeros(2, 2, R.D, device=DEV, dtype=torch.bfloat16)
    ws = native.Workspace(2, 4, 2, 30)
    active = torch.tensor([4, 0, 1, 2, 3], dtype=torch.int32, device=DEV)
    full = native.decode_attention_quant(q, c.k, c.v, c.scales, v0,
                                         torch.tensor([30, 1], dtype=torch.int32, device=DEV), active, workspace=ws)
    got = native.decode_attention_quant(q, c.k, c.v, c.scales, v0,
                                        torch.tensor([77, 0], dtype=torch.int32, device=DEV), active, workspace=ws)
    assert ws.device_error() == native.SR_DEVERR_SEQ_LEN and torch.equal(got, full)
    ws.clear_device_error()
    native.decode_attention_quant(q, c.k, c.v, c.scales, v0, torch.tensor([3, 3], dtype=torch.int32, device=DEV),
                                  torch.tensor([3, 0, 2, 1, 9], dtype=torch.int32, device=DEV), workspace=ws)
    assert ws.device_error() == native.SR_DEVERR_ACTIVE_LIST


@both
def test_far_positions_of_a_cache_over_4_gib(dtype):
    """Rows behind byte offset 2^32 and position 2^24: written, scanned and read
    back. All other rows are zero keys (logit 0) and zero values."""
    Lmax, Hkv, M = (1 << 24) + 3, 2, 4
    c = native.QuantCache(1, Hkv, Lmax, dtype)
    c.scales.fill_(1.0)
    x, y = rows((1, 3, Hkv, R.D), 4)[:, :, :, :], torch.randn(1, 3, Hkv, R.D, generator=gen(6), device=DEV)
    x = torch.randn(1, 3, Hkv, R.D, generator=gen(5), device=DEV).to(torch.bfloat16)
    y = y.to(torch.bfloat16)
    st = torch.tensor([Lmax - 3], dtype=torch.int32, device=DEV)
    native.kv_append_quant(x, y, st, torch.full_like(st, 3), c.k, c.v, c.scales)
    k, v = (torch.zeros(1, Hkv, 3, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    native.kv_dequant(c.k, c.v, c.scales, st, torch.full_like(st, 3), k, v)
    kc, ks = R.quantise(x[0].transpose(0, 1), dtype)
    vc, vs = R.quantise(y[0].transpose(0, 1), dtype)
    assert torch.equal(c.k[0, :, -3:].double(), kc) and torch.equal(c.v[0, :, -3:].double(), vc)
    kd, vd = kc * ks[..., None].double(), vc * vs[..., None].double()
    assert torch.allclose(k[0].double(), kd, rtol=2.0 ** -8, atol=0) and torch.allclose(v[0].double(), vd, rtol=2.0 ** -8, atol=0)
    # queries along the last keys, so that these hold most of the weight
    q = (4.0 * kd[:, 2:3] + 0.1 * torch.randn(Hkv, M, R.D, generator=gen(7), device=DEV)).to(torch.bfloat16).reshape(1, Hkv * M, R.D)
    sl = torch.tensor([Lmax], dtype=torch.int32, device=DEV)
    active = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    lse = torch.zeros(1, Hkv * M, device=DEV)
    out = native.decode_attention_quant(q, c.k, c.v, c.scales, v[:, :, 0].contiguous(), sl, active, lse=lse)
    for g in range(Hkv):
        h = slice(g * M, (g + 1) * M)
        s = q[0, h].double() @ kd[g].T / math.sqrt(R.D)
        e = torch.exp(s)
        tot = e.sum(-1, keepdim=True) + (Lmax - 3)
        o = e @ vd[g] / tot
        a = e @ vd[g].abs() / tot
        delta = 130 * R.HALF_F32 * (q[0, h].double().abs() @ kd[g].abs().T / math.sqrt(R.D)).amax(-1)
        # the sum of 2^24 ones in fp32: lanes, warps and splits add at most 2^14 of them in a row. Weights far
        # below the last row's may vanish, as in check_scan: fp16's smallest step is 2^-24, half of it is lost,
        # and the weights are scaled by 2^14, so three rows can lose 2^-39 of the largest weight each.
        under = 3 * 2.0 ** -39 * float(vd[g].abs().max())
        lim = R.bound(o, a, delta, R.HALF_F16, R.HALF_BF16, under) + 2.0 ** -10 * a
        err = (out[0, h].double() - o).abs()
        assert bool((err <= lim).all()), float((err / lim).max())
        assert ((lse[0, h].double() - torch.log(tot[:, 0])).abs() <= R.lse_bound(torch.log(tot[:, 0]), delta) + 2.0 ** -10).all()


class _BadStream:
    cuda_stream = "default"


def test_binding_refusals_on_the_gpu():
    """Every tensor's shape, type, layout and device is held against the cache's."""
    c = native.QuantCache(2, 4, 9)
    q = torch.zeros(2, 8, R.D, device=DEV, dtype=torch.bfloat16)
    v0 = torch.zeros(2, 4, R.D, device=DEV, dtype=torch.bfloat16)
    sl = torch.ones(2, dtype=torch.int32, device=DEV)
    act = torch.zeros(9, dtype=torch.int32, device=DEV)
    good = dict(q=q, k_cache=c.k, v_cache=c.v, kv_scales=c.scales, v0=v0, seq_lens=sl, active_list=act)
    native.decode_attention_quant(*good.values())
    bad = dict(q=[q[:1], q.float(), q.cpu(), q[:, :7]], v_cache=[c.v[:, :, :8], c.v.view(torch.int8), c.v.cpu()],
               kv_scales=[c.scales[..., :1], c.scales.double(), c.scales.transpose(0, 1)], v0=[v0[:, :3], v0.float()],
               seq_lens=[sl[:1], sl.long()], active_list=[act[:8], act.float()])
    for name, tensors in bad.items():
        for t in tensors:
            with pytest.raises((ValueError, native.SinkRouterError)):
                native.decode_attention_quant(*(t if n == name else x for n, x in good.items()))
    x = torch.zeros(2, 3, 4, R.D, device=DEV, dtype=torch.bfloat16)
    wide = torch.zeros(2, 3, 4, R.D + 4, device=DEV, dtype=torch.bfloat16)[..., :R.D]  # rows not 16-byte aligned
    for k_new in (x[:, :, :3], x.float(), x.transpose(1, 2), wide):
        with pytest.raises((ValueError, native.SinkRouterError)):
            native.kv_append_quant(k_new, x, sl, sl, c.k, c.v, c.scales)
    with pytest.raises(native.SinkRouterError):
        native.kv_append_quant(x, x, sl, sl, c.k, c.v, c.scales, k0=v0)  # k0 without v0
    with pytest.raises(ValueError, match="kv_scales"):
        native.kv_append_quant(x, x, sl, sl, c.k, c.v, None)
    cs = torch.zeros(20, 64, device=DEV)
    kn = torch.zeros(2, 4, R.D, device=DEV, dtype=torch.bfloat16)
    bf = torch.zeros(2, 4, 9, R.D, device=DEV, dtype=torch.bfloat16)
    for cache, sc, tables, tau, off in ((bf, c.scales, cs, 0.6, 0), (c.k, None, cs, 0.6, 0), (c.k, c.scales, cs[:, :32], 0.6, 0),
                                        (c.k, c.scales, cs, "x", 0), (c.k, c.scales, cs, math.nan, 0),
                                        (c.k, c.scales, cs, 0.6, -1), (c.k, c.scales, cs, 0.6, 2 ** 40),
                                        (c.k, c.scales, cs, 0.6, 0.5), (bf.float(), None, cs, 0.6, 0)):
        with pytest.raises((ValueError, native.SinkRouterError)):
            native.rope_append_route_kv(q, kn, kn, tables, tables, sl, cache, cache, sc, v0, v0, tau, pos_offset=off)
    for bad in (dict(q_out=q[:1]), dict(route_mask=act), dict(active_list=act[:3]), dict(seq_lens_out=sl.long()),
                dict(device_error=sl)):
        with pytest.raises(ValueError):
            native.rope_append_route_kv(q, kn, kn, cs, cs, sl, c.k, c.v, c.scales, v0, v0, 0.6, **bad)
    with pytest.raises(ValueError):
        native.decode_attention_quant(*good.values(), stream=_BadStream)
    assert native.kv_append_quant(x[:, :0], x[:, :0], sl, sl, c.k, c.v, c.scales)[0] is c.k  # no token: nothing to do
    torch.cuda.synchronize()
    assert not c.scales.any()


# ---- together ----------------------------------------------------------------------------

@both
def test_prefill_then_decode_steps(dtype):
    """A prompt is written in two chunks, then tokens are appended and attended to,
    each step against 64 bits on the cache that the definitions give."""
    B, Hkv, M, Lmax = 2, 4, 4, 96
    Hq = Hkv * M
    prompt = [50, 33]
    k, v = rows((B, 50, Hkv, R.D), 3), torch.randn(B, 50, Hkv, R.D, generator=gen(4), device=DEV).to(torch.bfloat16)
    k = torch.randn(B, 50, Hkv, R.D, generator=gen(5), device=DEV).to(torch.bfloat16)
    c = native.QuantCache(B, Hkv, Lmax, dtype)
    k0, v0 = (torch.zeros(B, Hkv, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    n1 = torch.tensor([30, 30], dtype=torch.int32, device=DEV)
    n2 = torch.tensor([n - 30 for n in prompt], dtype=torch.int32, device=DEV)
    native.kv_append_quant(k[:, :30], v[:, :30], torch.zeros_like(n1), n1, c.k, c.v, c.scales, k0, v0)
    native.kv_append_quant(k[:, 30:], v[:, 30:], n1, n2, c.k, c.v, c.scales, k0, v0)
    assert torch.equal(k0, k[:, 0]) and torch.equal(v0, v[:, 0])
    seq = (n1 + n2).clone()
    cs, sn = inputs.rope_tables(Lmax, device=DEV)
    dec = native.QuantDecoder(B, Hq, Hkv, Lmax)
    keys, values = ([[x[b, :prompt[b]].transpose(0, 1)] for b in range(B)] for x in (k, v))
    o = oracle.load()
    dummy = torch.zeros(B, Hkv, Lmax, R.D, dtype=torch.bfloat16)
    for step in range(4):
        q, kn, vn = inputs.make_projections(B, Hq, Hkv, seed=40 + step, device=DEV)
        before = seq.cpu()
        out = dec.append_step(q, kn, vn, cs, sn, c, k0, v0, seq, TAU)
        ref = o.rope_append(q, kn, vn, cs, sn, before, dummy, dummy, k0, v0)
        assert torch.equal(dec.q.cpu().view(torch.int16), ref[1].view(torch.int16))
        assert torch.equal(seq.cpu(), before + 1)
        for b in range(B):
            keys[b].append(ref[2][b, :, before[b]].to(DEV)[:, None])
            values[b].append(vn[b][:, None])
        mask = dec.route_mask.view(B, Hkv).tolist()
        for b in range(B):
            kc, ks = R.quantise(torch.cat(keys[b], 1), dtype)
            vc, vs = R.quantise(torch.cat(values[b], 1), dtype)
            for g in range(Hkv):
                h = slice(g * M, (g + 1) * M)
                if mask[b][g]:
                    assert torch.equal(out[b, h], v0[b, g].expand(M, -1))
                    continue
                vd = vc[g] * vs[g][:, None].double()
                oo, _, a, delta = R.attention(dec.q[b, h], kc[g] * ks[g][:, None].double(), vd, vd.shape[0])
                under = vd.shape[0] * 2.0 ** -39 * float(vd.abs().max())
                assert ((out[b, h].double() - oo).abs() <= R.bound(oo, a, delta, R.HALF_F16, R.HALF_BF16, under)).all()
    assert dec.workspace.device_error() == 0


@both
@pytest.mark.parametrize("B,Hkv,M", [(1, 8, 4), (40, 8, 2)], ids=["few", "many"])
def test_captured_append_steps_advance(B, Hkv, M, dtype):
    """append_step in a CUDA graph: every replay takes the next slot of what the
    lengths then are, like eager steps on a second cache; a full cache is reported and
    left alone."""
    Lmax, Hq = 24, Hkv * M
    cs, sn = inputs.rope_tables(Lmax, device=DEV)
    proj = [inputs.make_projections(B, Hq, Hkv, seed=70 + i, device=DEV) for i in range(5)]
    side = []
    for _ in range(2):
        c = native.QuantCache(B, Hkv, Lmax, dtype)
        k0, v0 = (torch.zeros(B, Hkv, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        seq = torch.tensor([(5 * b) % 20 for b in range(B)], dtype=torch.int32, device=DEV)
        fill = torch.randn(B, Lmax, Hkv, R.D, generator=gen(3), device=DEV).to(torch.bfloat16)
        native.kv_append_quant(fill, fill, torch.zeros_like(seq), seq, c.k, c.v, c.scales, k0, v0)
        side.append((c, k0, v0, seq, native.QuantDecoder(B, Hq, Hkv, Lmax), torch.zeros(1, dtype=torch.int32, device=DEV)))
    q, kn, vn = (torch.empty_like(x) for x in proj[0])
    step = lambda s, x: s[4].append_step(*x, cs, sn, s[0], s[1], s[2], s[3], TAU, device_error=s[5])  # noqa: E731
    for x in (q, kn, vn):
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    warm = [t.clone() for t in (side[0][0].k.view(torch.uint8), side[0][0].v.view(torch.uint8), side[0][0].scales,
                                side[0][1], side[0][2], side[0][3])]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(side[0], (q, kn, vn))
    torch.cuda.current_stream().wait_stream(stream)
    with torch.cuda.graph(graph):
        step(side[0], (q, kn, vn))
    for t, w in zip((side[0][0].k.view(torch.uint8), side[0][0].v.view(torch.uint8), side[0][0].scales, side[0][1],
                     side[0][2], side[0][3]), warm):
        t.copy_(w)
    side[0][5].zero_()
    for x in proj:
        for dst, src in zip((q, kn, vn), x):
            dst.copy_(src)
        graph.replay()
        want = step(side[1], x)
        torch.cuda.synchronize()
        assert torch.equal(side[0][4].out, want)
        for a, b in zip(side[0][1:4], side[1][1:4]):
            assert torch.equal(a, b)
        assert torch.equal(side[0][0].k.view(torch.uint8), side[1][0].k.view(torch.uint8))
        assert torch.equal(side[0][0].scales, side[1][0].scales)
    assert int(side[0][5]) == int(side[1][5]) == (native.SR_DEVERR_APPEND_SLOT if B > 4 and max((5 * b) % 20 for b in range(B)) + 5 > Lmax else 0)
    assert int(side[0][3].max()) <= Lmax


def test_scan_of_units_that_are_one_split_each():
    """Many short units (a split each, written without a partial) against the same
    units cut into three splits: the same attention inside both bounds, and bf16 out
    equal to the rounded fp32 partial."""
    B, Hkv, M, Lmax = 60, 4, 2, 300
    lens = [1 + (37 * b) % Lmax for b in range(B)]
    for dtype in R.DTYPES:
        c = filled_cache(B, Hkv, Lmax, lens, dtype, 31)
        q = torch.randn(B, Hkv * M, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
        v0 = torch.randn(B, Hkv, R.D, generator=gen(2), device=DEV).to(torch.bfloat16)
        mask = torch.rand(B, Hkv, generator=gen(3), device=DEV) < 0.2
        for ns in (0, 1, 3):
            out, lse, o = scan(q, c, v0, lens, mask, ns)
            check_scan(q, c, v0, lens, mask.tolist(), out, lse, o)
            assert torch.equal(out, o.to(torch.bfloat16))


@both
@pytest.mark.parametrize("B,Hkv,M,Lmax,ns", [
    (33, 1, 4, 67, 0),     # more than 32 units
    (1, 1, 4, 40193, 0),   # the last share ends with a tile of one row
    (1, 1, 8, 1001, 3),    # forced splits of two tiles
    (1, 5, 4, 4099, 1),    # one split of 17 tiles
    (3, 11, 1, 513, 5),    # 33 units, forced splits
    (1, 3, 2, 257, 1),     # the last pair alone in the last tile
])
def test_scan_reads_the_last_pair_of_an_odd_count(B, Hkv, M, Lmax, ns, dtype):
    """An odd number of scale pairs leaves the last one without a neighbour for the
    16-byte copy. All sequences full, the last unit active, the last position of every
    unit aligned with its queries and its value scale eight times the others'; several
    times over, with other values in between."""
    assert B * Hkv * Lmax % 2 == 1
    lens = [Lmax] * B
    v0 = torch.randn(B, Hkv, R.D, generator=gen(2), device=DEV).to(torch.bfloat16)
    mask = torch.zeros(B, Hkv, dtype=torch.bool, device=DEV)
    mask[0, 0] = True
    for seed in (11, 12, 13):
        c = filled_cache(B, Hkv, Lmax, lens, dtype, seed)
        q = torch.randn(B, Hkv, M, R.D, generator=gen(seed + 7), device=DEV)
        last = c.k[:, :, -1].float() * c.scales[:, :, -1, :1]
        q = (0.3 * q + 2.0 * last[:, :, None] / last[:, :, None].norm(dim=-1, keepdim=True)).to(torch.bfloat16)
        c.scales[:, :, -1, 0] *= 4.0
        c.scales[:, :, -1, 1] *= 8.0
        out, lse, o = scan(q.reshape(B, Hkv * M, R.D), c, v0, lens, mask, ns)
        check_scan(q.reshape(B, Hkv * M, R.D), c, v0, lens, mask.tolist(), out, lse, o)


@pytest.mark.parametrize("kind", ["bf16", *R.IDS])
@pytest.mark.parametrize("M", [1, 4, 8])
@pytest.mark.parametrize("L,bad,ns", [
    (33, range(32, 33), 0), (65, range(64, 65), 0), (129, range(128, 129), 0),  # a warp's only row
    (300, range(0, 128), 0),             # all rows of a warp, or of several
    (4, range(3, 4), 4), (4, range(0, 1), 4),         # a split's only row
    (64, range(0, 25), 64), (64, range(30, 64), 64),  # a whole batch of the merge
    (5000, range(4992, 5000), 0),        # the end of the last share
    (1, range(0, 1), 0), (70, range(0, 70), 7),       # nothing but NaN
], ids=lambda x: f"{x.start}to{x.stop}" if isinstance(x, range) else str(x))
def test_nan_keys_reach_the_result_whatever_shares_their_rows(L, bad, ns, M, kind):
    """NaN logits leave the running maximum as it is, so a warp or a split that holds
    nothing else has a maximum of -inf: its NaN must not be taken for a part without
    rows. The other unit of the launch stays finite."""
    q = torch.randn(1, 2 * M, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    v0 = torch.randn(1, 2, R.D, generator=gen(2), device=DEV).to(torch.bfloat16)
    sl = torch.tensor([L], dtype=torch.int32, device=DEV)
    active = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    lse = torch.zeros(1, 2 * M, device=DEV)
    if kind == "bf16":
        k, v = (torch.randn(1, 2, L, R.D, generator=gen(i), device=DEV).to(torch.bfloat16) for i in (3, 4))
        k[0, 1, bad.start:bad.stop, 17] = math.nan
        out = native.decode_attention(q, k, v, None, v0, sl, active, n_splits=ns, lse=lse)
        o, z = native.decode_attention_partial(q, k, v, None, v0, sl, active, n_splits=ns)
    else:
        c = filled_cache(1, 2, L, [L], R.DTYPES[R.IDS.index(kind)], 3)
        c.scales[0, 1, bad.start:bad.stop, 0] = math.nan
        out = native.decode_attention_quant(q, c.k, c.v, c.scales, v0, sl, active, n_splits=ns, lse=lse)
        o, z = native.decode_attention_quant_partial(q, c.k, c.v, c.scales, v0, sl, active, n_splits=ns)
    for t in (out, o, lse, z):
        assert torch.isfinite(t[0, :M]).all() and torch.isnan(t[0, M:]).all()


@both
@pytest.mark.parametrize("exp", [-120.0, 60.0, 125.9, 126.2, 127.0, 127.9])
def test_scan_takes_value_scales_to_the_end_of_fp32(exp, dtype):
    """Codes of -1, 0 and 1 under scales up to nearly 2^128: one position with the
    largest scale holds nearly all the weight (so that no sum passes fp32's end), the
    others' scales are 2^9 below it."""
    n = 200
    c = filled_cache(1, 2, n, [n], dtype, 3)
    q = torch.randn(1, 8, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    v0 = torch.zeros(1, 2, R.D, device=DEV, dtype=torch.bfloat16)
    c.v.copy_(torch.randint(-1, 2, c.v.shape, generator=gen(3), device=DEV).float().to(dtype))
    c.scales[..., 1] = 2.0 ** (exp - 9)
    key = c.k[0, :, 77].float() * c.scales[0, :, 77, :1]
    q = (q.view(2, 4, R.D).float() * 0.1 + 4 * key[:, None] / key[:, None].norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    c.scales[0, :, 77, 0] *= 40.0
    c.scales[0, :, 77, 1] = 2.0 ** exp
    mask = torch.zeros(1, 2, dtype=torch.bool, device=DEV)
    out, lse, o = scan(q.reshape(1, 8, R.D), c, v0, [n], mask)
    check_scan(q.reshape(1, 8, R.D), c, v0, [n], mask.tolist(), out, lse, o)
    big = float(out.double().abs().max())
    assert 2.0 ** (exp - 0.1) < big <= 2.0 ** (exp + 0.01)


@both
def test_append_quant_takes_the_largest_token_count(dtype):
    """T = 2^31 - 1 (a view of one token repeated): the blocks of four tokens round it
    up past 2^31."""
    c = sentinel_cache(1, 2, 8, dtype)
    x = rows((1, 1, 2, R.D), 3)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    many = x.expand(1, 2 ** 31 - 1, 2, R.D)
    native.kv_append_quant(many, many, z + 1, z + 3, c.k, c.v, c.scales, device_error=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert_rows(c.k[0, :, 1:4], c.scales[0, :, 1:4, 0], x[0, 0, :, None].expand(2, 3, R.D), dtype, "rows")
    assert (c.scales[0, :, [0, 4, 5, 6, 7]] == -7.0).all()


def test_a_workspace_of_another_device_is_refused(monkeypatch):
    """Its memory may not be reachable from the call's device. One GPU: the workspace
    says that it is elsewhere."""
    c = native.QuantCache(2, 4, 9)
    q = torch.zeros(2, 8, R.D, device=DEV, dtype=torch.bfloat16)
    v0 = torch.zeros(2, 4, R.D, device=DEV, dtype=torch.bfloat16)
    sl, act = torch.ones(2, dtype=torch.int32, device=DEV), torch.zeros(9, dtype=torch.int32, device=DEV)
    ws, pws = native.Workspace(2, 8, 4, 9), native.PrefixWorkspace(2, 8, 4, 9)
    assert ws.device_index == pws.device_index == q.get_device()
    monkeypatch.setattr(ws, "device_index", 7)
    monkeypatch.setattr(pws, "device_index", 7)
    mask = torch.zeros(8, dtype=torch.uint8, device=DEV)
    kp = torch.zeros(4, 9, R.D, device=DEV, dtype=torch.bfloat16)
    for call, w in ((native.decode_attention_quant, ws), (native.decode_attention_quant_partial, ws)):
        with pytest.raises(ValueError, match="cuda:7"):
            call(q, c.k, c.v, c.scales, v0, sl, act, workspace=w)
    for call in (native.prefix_attention, native.prefix_attention_partial):
        with pytest.raises(ValueError, match="cuda:7"):
            call(q, kp, kp, 9, v0, mask, workspace=pws)


def test_calls_in_a_row_see_what_the_one_before_wrote():
    """Chains without a host wait in which a call's inputs are what the previous call's
    kernel wrote, while its own kernel may already be resident: position-0 rows into
    routing and the sink bypass, lengths into a read-back, a partial into the
    combination. Fresh values in the same buffers every time."""
    B, Hkv, M, L = 3, 8, 4, 6
    Hq = Hkv * M
    c = native.QuantCache(B, Hkv, L)
    k0, v0 = (torch.zeros(B, Hkv, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    zero, n = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    mask = torch.zeros(B * Hkv, dtype=torch.uint8, device=DEV)
    active = torch.zeros(1 + B * Hkv, dtype=torch.int32, device=DEV)
    ws = native.Workspace(B, Hq, Hkv, L)
    out = torch.zeros(B, Hq, R.D, device=DEV, dtype=torch.bfloat16)
    ko, vo = (torch.zeros(B, Hkv, L, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    cs, sn = inputs.rope_tables(L, device=DEV)
    part = torch.zeros(2, B * Hq * R.D, device=DEV)
    lse = torch.zeros(2, B * Hq * R.D, device=DEV)
    joined = torch.zeros_like(out)
    rounds = 40
    x = torch.randn(rounds, 2, B, 1, Hkv, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    q = torch.randn(rounds, B, Hkv, M, R.D, generator=gen(2), device=DEV)
    near = torch.rand(rounds, B, Hkv, 1, 1, generator=gen(3), device=DEV) < 0.5
    q = torch.where(near, x[:, 0, :, 0, :, None].float() + 0.1 * q, q).to(torch.bfloat16).reshape(rounds, B, Hq, R.D)
    lens = torch.randint(1, L, (rounds, B), generator=gen(4), device=DEV, dtype=torch.int32)
    one = torch.ones_like(n)
    seen = []
    torch.cuda.synchronize()
    for i in range(rounds):
        native.kv_append_quant(x[i, 0], x[i, 1], zero, one, c.k, c.v, c.scales, k0, v0)
        native.route(q[i], k0, TAU, mask, active)
        native.decode_attention_quant_partial(q[i], c.k, c.v, c.scales, v0, one, active, part[0].view(B, Hq, R.D),
                                              lse[0, :B * Hq].view(B, Hq), workspace=ws)
        native.combine_partials(part, lse, B * Hq * R.D, 1, B, Hq, joined)
        native.decode_attention_quant(q[i], c.k, c.v, c.scales, v0, one, active, out, workspace=ws)
        native.rope_append_route_kv(q[i], x[i, 0, :, 0], x[i, 1, :, 0], cs, sn, lens[i], c.k, c.v, c.scales, k0, v0, TAU,
                                    seq_lens_out=n)
        native.kv_dequant(c.k, c.v, c.scales, zero, n, ko, vo)
        seen.append([t.clone() for t in (mask, out, joined, n, ko, vo)])
    torch.cuda.synchronize()
    for i, (m, o, j, nn, k, v) in enumerate(seen):
        assert torch.equal(m.view(B, Hkv), near[i, ..., 0, 0].to(torch.uint8)) and torch.equal(nn, lens[i] + 1)
        assert torch.equal(o, j)
        kc, ks = R.quantise(x[i, :, :, 0], R.E4M3)  # [2, B, Hkv, 128]
        row = (kc * ks[..., None].double()).to(torch.bfloat16)
        for b in range(B):
            for g in range(Hkv):  # one position: its value row, or the position-0 value
                want = x[i, 1, b, 0, g] if near[i, b, g] else row[1, b, g]
                assert torch.equal(o.view(B, Hkv, M, R.D)[b, g], want.expand(M, -1))
            assert torch.equal(v[b, :, int(nn[b]) - 1], row[1, b])


def spread(n, count):
    """About `count` indices over [0, n), the last among them."""
    return sorted({*range(0, n, max(1, n // count)), n - 1})


@pytest.mark.parametrize("ns", [0, 2])
@pytest.mark.parametrize("B,Hkv,M,Lmax", [(16384, 1, 1, 3), (2048, 8, 8, 70), (5000, 1, 8, 130)])
def test_scan_of_the_largest_launches(B, Hkv, M, Lmax, ns):
    """Up to the most units that a launch takes, more sequences than the length table
    holds, an odd number of scale pairs; a spread of sequences is checked."""
    lens = [1 + (7 * b) % Lmax for b in range(B)]
    c = filled_cache(B, Hkv, Lmax, lens, R.E4M3, 3, poison=False)
    q = torch.randn(B, Hkv * M, R.D, generator=gen(1), device=DEV).to(torch.bfloat16)
    v0 = torch.randn(B, Hkv, R.D, generator=gen(2), device=DEV).to(torch.bfloat16)
    mask = torch.rand(B, Hkv, generator=gen(3), device=DEV) < 0.3
    out, lse, o = scan(q, c, v0, lens, mask, ns)
    at = spread(B, 40)
    part = native.QuantCache(len(at), Hkv, Lmax)
    for to, x in ((part.k, c.k), (part.v, c.v)):
        to.view(torch.uint8).copy_(x.view(torch.uint8)[at])
    part.scales.copy_(c.scales[at])
    check_scan(q[at], part, v0[at], [lens[i] for i in at], mask[at].tolist(), out[at], lse[at], o[at])


@both
@pytest.mark.parametrize("B,Hkv,M", [(2048, 8, 8), (16384, 1, 1), (33, 8, 8), (12, 4, 8), (48, 1, 8)])
def test_append_of_the_largest_launches(B, Hkv, M, dtype):
    """The 8-bit append in its three spreads, up to the most units, against the bf16 one:
    the same query, routing and lengths, and its rotated key quantised."""
    Lmax = 5
    c = native.QuantCache(B, Hkv, Lmax, dtype)
    q, kn, vn = inputs.make_projections(B, Hkv * M, Hkv, seed=1, device=DEV)
    cs, sn = inputs.rope_tables(Lmax, device=DEV)
    k0, v0 = (torch.randn(B, Hkv, R.D, generator=gen(i), device=DEV).to(torch.bfloat16) for i in (1, 2))
    seq = torch.tensor([(3 * b) % Lmax for b in range(B)], dtype=torch.int32, device=DEV)
    at = seq.long()
    kb, vb = (torch.zeros(B, Hkv, Lmax, R.D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    k0b, v0b, seqb = k0.clone(), v0.clone(), seq.clone()
    q1, m1, a1 = native.rope_append_route_kv(q, kn, vn, cs, sn, seq, c.k, c.v, c.scales, k0, v0, TAU)
    q2, m2, a2 = native.rope_append_route(q, kn, vn, cs, sn, seqb, kb, vb, k0b, v0b, TAU)
    n = int(a2[0])
    for x, y in ((q1, q2), (m1, m2), (a1[:1 + n], a2[:1 + n]), (seq, seqb), (k0, k0b), (v0, v0b)):
        assert torch.equal(x, y)
    i = torch.arange(B, device=DEV)
    for codes, part, rows_of in ((c.k, 0, kb), (c.v, 1, vb)):
        assert_rows(codes.view(torch.uint8)[i, :, at].view(dtype), c.scales[i, :, at][..., part], rows_of[i, :, at], dtype,
                    "appended rows")
