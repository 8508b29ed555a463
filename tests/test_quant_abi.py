"""Host-side refusals of the 8-bit cache and shared-prefix entry points: nothing is
launched, so these run without a GPU. Also the binding's own checks of shapes."""
import ctypes

import pytest
import torch

from kv_cache_routing_sr_b200 import build, native, shared_prefix

FAKE = 0x10000  # aligned, never dereferenced: validation fails before any launch
INV, UNS, WS = native.SR_ERR_INVALID_ARG, native.SR_ERR_UNSUPPORTED, native.SR_ERR_WORKSPACE
BAD_DIMS = [(dict(d=64), UNS), (dict(Hq=24), UNS), (dict(B=4097), UNS), (dict(B=0), INV), (dict(Hq=30), INV),
            (dict(L=0), INV)]


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return native.load()


def dims(B=1, Hq=32, Hkv=8, d=128, L=4096):
    return native.Dims(B, Hq, Hkv, d, L)


def caller(lib, name, order, fixed):
    """A call of an entry point with any argument replaced by keyword."""
    def call(dims=dims(), **kw):
        args = [kw.get(n, fixed.get(n, FAKE)) for n in order]
        args = [ctypes.c_float(a) if n == "tau" else ctypes.byref(a) if isinstance(a, ctypes.Structure) else a
                for n, a in zip(order, args)]
        return getattr(lib, name)(ctypes.byref(dims), *args, None)
    return call


def strides(b=8, t=8, h=8):
    return native.RowStrides(b, t, h)


def refuses(call, cases):
    for kw, expect in cases:
        assert call(**kw) == expect, kw


def common(call, pointers, aligned16, aligned4, extra=()):
    refuses(call, [({n: None}, INV) for n in pointers])
    refuses(call, [({n: FAKE + 8}, INV) for n in aligned16])
    refuses(call, [({n: FAKE + 2}, INV) for n in aligned4])
    refuses(call, [(dict(dims=dims(**d)), e) for d, e in BAD_DIMS])
    refuses(call, extra)


def test_kv_append_quant(lib):
    call = caller(lib, "sr_kv_append_quant",
                  ["kv", "T", "k", "ks", "v", "vs", "start", "n", "kc", "vc", "sc", "k0", "v0", "err"],
                  dict(kv=1, T=4, ks=strides(), vs=strides(), err=None))
    common(call, ["k", "ks", "v", "vs", "start", "n", "kc", "vc", "sc", "k0", "v0"], ["k", "v", "kc", "vc", "sc", "k0", "v0"],
           ["start", "n", "err"],
           [(dict(kv=0), INV), (dict(kv=3), INV), (dict(kv=-1), INV), (dict(T=0), INV), (dict(ks=strides(b=4)), INV),
            (dict(vs=strides(t=12)), INV), (dict(vs=strides(h=-1)), INV)])


def test_kv_dequant(lib):
    call = caller(lib, "sr_kv_dequant", ["kv", "T", "kc", "vc", "sc", "start", "n", "ko", "vo", "err"],
                  dict(kv=2, T=4, err=None))
    common(call, ["kc", "vc", "sc", "start", "n", "ko", "vo"], ["kc", "vc", "sc", "ko", "vo"], ["start", "n", "err"],
           [(dict(kv=0), INV), (dict(kv=7), INV), (dict(T=0), INV), (dict(T=-5), INV)])


def test_rope_append_route_kv(lib):
    rows = ["q", "kn", "vn", "cos", "sin", "kc", "vc", "k0", "v0", "qo"]
    call = caller(lib, "sr_rope_append_route_kv",
                  ["kv", "off", "q", "kn", "vn", "cos", "sin", "mp", "sl", "slo", "kc", "vc", "sc", "k0", "v0", "tau", "qo",
                   "mask", "act", "err"], dict(kv=1, off=0, mp=64, tau=0.6, err=None))
    common(call, rows + ["sl", "slo", "mask", "act", "sc"], rows + ["sc"], ["sl", "slo", "act", "err"],
           [(dict(kv=0), INV), (dict(kv=0, sc=None, mp=0), INV), (dict(kv=5), INV), (dict(off=-1), INV), (dict(mp=0), INV),
            (dict(tau=float("nan")), INV)])


@pytest.mark.parametrize("partial", [False, True])
def test_decode_attention_quant(lib, partial):
    outs = ["o", "lse"]
    call = caller(lib, "sr_decode_attention_quant" + ("_partial" if partial else ""),
                  ["kv", "q", "kc", "vc", "sc", "v0", "sl", "act", "ns", *outs, "ws", "wsb"], dict(kv=1, ns=0, wsb=1 << 30))
    need = native.workspace_bytes(1, 32, 8, 4096)
    common(call, ["q", "kc", "vc", "sc", "v0", "sl", "act", "o"] + (["lse"] if partial else []),
           ["q", "kc", "vc", "sc", "v0", "o"], ["sl", "act", "lse"],
           [(dict(kv=0), INV), (dict(kv=9), INV), (dict(ns=-1), INV), (dict(ns=native.SR_MAX_SPLITS + 1), INV),
            (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(wsb=need - 1), WS)])


def test_splits_by_unit_belong_to_the_partial_form(lib):
    order = ["q", "kc", "vc", "k0", "v0", "sl", "act", "ns"]
    part = caller(lib, "sr_decode_attention_partial", [*order, "o", "lse", "ws", "wsb"], dict(ws=None, wsb=1 << 30))
    whole = caller(lib, "sr_decode_attention", [*order, "o", "ws", "wsb"], dict(ws=None, wsb=1 << 30))
    # the workspace is looked at after the splits
    refuses(part, [(dict(ns=native.SPLITS_BY_UNIT), WS), (dict(ns=0), WS), (dict(ns=-2), INV)])
    refuses(whole, [(dict(ns=native.SPLITS_BY_UNIT), INV), (dict(ns=0), WS)])


@pytest.mark.parametrize("partial", [False, True])
def test_prefix_attention(lib, partial):
    order = ["Lp", "q", "k", "v", "v0", "mask"] + ([] if partial else ["os", "ls"]) + ["o", "lse", "ws", "wsb"]
    call = caller(lib, "sr_prefix_attention" + ("_partial" if partial else ""), order, dict(Lp=100, wsb=1 << 40))
    need = native.prefix_workspace_bytes(1, 32, 8, 4096)
    assert need % 256 == 0
    extra = [(dict(Lp=-1), INV), (dict(Lp=4097), INV), (dict(ws=None), WS), (dict(ws=FAKE + 16), WS),
             (dict(wsb=need - 1), WS)]
    if partial:
        extra.append((dict(lse=None), INV))
    else:  # both parts of the suffix, or none
        extra += [(dict(os=None), INV), (dict(ls=None), INV), (dict(os=FAKE + 8), INV), (dict(ls=FAKE + 2), INV)]
    common(call, ["q", "k", "v", "v0", "mask", "o"], ["q", "k", "v", "v0", "o"], ["lse"], extra)
    for d, _ in BAD_DIMS:
        assert lib.sr_prefix_workspace_bytes(ctypes.byref(dims(**d))) == 0
    assert lib.sr_prefix_workspace_bytes(None) == 0


def test_binding_refuses_cpu_tensors_and_wrong_kinds(lib):
    """What the binding refuses before it would look at a device: CPU tensors, things
    that are no tensors, caches of another type or rank, scales that do not belong."""
    i32, bf16 = torch.int32, torch.bfloat16
    k = torch.zeros(2, 4, 9, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc, n = torch.zeros(2, 4, 9, 2), torch.zeros(2, dtype=i32)
    b = torch.zeros(2, 4, 9, 128, dtype=bf16)
    with pytest.raises(ValueError, match="CUDA"):
        native.kv_dequant(k, k, sc, n, n, b, b)
    with pytest.raises(ValueError, match="tensor"):
        native.kv_dequant(None, k, sc, n, n, b, b)
    with pytest.raises(ValueError, match="CUDA"):
        native.kv_append_quant(b, b, n, n, k, k, sc)
    with pytest.raises(ValueError, match="CUDA"):
        native.prefix_attention(torch.zeros(2, 8, 128, dtype=bf16), b[0], b[0], 3, torch.zeros(2, 4, 128, dtype=bf16),
                                torch.zeros(8, dtype=torch.uint8), workspace=_FakeWorkspace)
    with pytest.raises(ValueError, match="CUDA"):
        native.decode_attention_quant(torch.zeros(2, 8, 128, dtype=bf16), k, k, sc, b[:, :, 0].contiguous(), n, n,
                                      workspace=_FakeWorkspace)
    with pytest.raises(ValueError, match="8-bit"):
        native.QuantCache(1, 1, 1, torch.float16, device="cpu")
    assert shared_prefix.SharedPrefixDecoder


class _FakeWorkspace:
    ptr, nbytes = FAKE, 1 << 30


@pytest.fixture
def unloaded(monkeypatch):
    """native as in a process that has loaded nothing yet; what would be compiled."""
    made = []
    monkeypatch.setattr(native, "_lib", None)
    monkeypatch.setattr(native, "_bound", None)
    monkeypatch.setattr(build, "build", lambda *a, **k: made.append("library"))
    monkeypatch.setattr(build, "build_binding", lambda *a, **k: made.append("binding"))
    return made


def test_the_library_loads_without_the_binding(lib, unloaded, monkeypatch, tmp_path):
    """The entry points that ctypes serves need no binding, no compiler and no headers."""
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_sr_binding.so"))
    monkeypatch.setenv("SINKROUTER_LIBRARY", build.LIBRARY)
    assert native.load().sr_status_string(0) == b"SR_OK" and unloaded == []
    assert native.workspace_bytes(1, 32, 8, 4096) > 0 and unloaded == []


def test_only_the_binding_is_compiled_where_only_it_is_missing(lib, unloaded, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_sr_binding.so"))
    native._loaded()
    assert unloaded == ["binding"]
    native._loaded()
    assert unloaded == ["binding"]


def test_a_failed_compile_of_the_binding_says_so(lib, unloaded, monkeypatch, tmp_path):
    def fails(*a):
        raise RuntimeError("no g++")
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_sr_binding.so"))
    monkeypatch.setattr(build, "build_binding", fails)
    with pytest.raises(RuntimeError, match="_sr_binding.so.*no g"):
        native.kv_dequant(*[None] * 7)
    assert native.load() is not None  # the rest still works


def test_a_binding_of_another_torch_is_noticed(lib, unloaded, monkeypatch):
    assert build.binding_current() and not build.needs_build()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    assert not build.binding_current() and build.needs_build()


# ---- the decoders' own checks: nothing is launched, appended or routed before they pass ----

@pytest.fixture
def launched(monkeypatch):
    """Names of the entry points that a step has reached."""
    calls = []
    for name in ("route", "rope_append_route_kv", "decode_attention_partial", "decode_attention_quant",
                 "decode_attention_quant_partial", "prefix_attention"):
        monkeypatch.setattr(native, name, lambda *a, _n=name, **k: calls.append(_n))
    return calls


def bare(cls, B, Hq, Hkv, L):
    """A decoder of CPU buffers, as far as the checks look at it."""
    d = object.__new__(cls)
    d.shape = (B, Hq, Hkv, L)
    d.out = d.q = torch.zeros(B, Hq, 128, dtype=torch.bfloat16)
    d.route_mask = d.active_list = None
    d.workspace = type("W", (), dict(nbytes=native.workspace_bytes(B, Hq, Hkv, L), ptr=FAKE))
    return d


def half(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def shifted(*shape):
    """bf16, contiguous, two bytes off a 16-byte boundary."""
    n = torch.Size(shape).numel()
    return half(n + 16)[1:n + 1].view(shape)


def test_quant_decoder_refuses_tensors_of_another_shape_before_it_launches(lib, launched):
    B, Hq, Hkv, L = 2, 8, 4, 9
    dec = bare(native.QuantDecoder, B, Hq, Hkv, L)
    cache = native.QuantCache(B, Hkv, L, device="cpu")
    lens = torch.ones(B, dtype=torch.int32)
    good = dict(q=half(B, Hq, 128), k0=half(B, Hkv, 128), n_splits=0)
    bad = dict(q=[half(B + 1, Hq, 128), half(1, Hq, 128), half(B, 16, 128), half(B, Hq, 64), half(B, Hq, 128).float(),
                  half(Hq, B, 128).transpose(0, 1), shifted(B, Hq, 128), half(B, Hq, 128).to("meta")],
               k0=[half(B + 1, Hkv, 128), half(B, 8, 128), half(B, Hkv, 128).float()],
               n_splits=[-1, native.SR_MAX_SPLITS + 1, 2000])

    def steps(q, k0, n_splits):
        yield lambda: dec.step(q, cache, k0, good["k0"], lens, 0.6, n_splits)
        yield lambda: dec.append_step(q, good["k0"], good["k0"], half(L, 64), half(L, 64), cache, k0, good["k0"], lens, 0.6,
                                      n_splits)
    for name, values in bad.items():
        for v in values:
            for call in steps(**{**good, name: v}):
                with pytest.raises((ValueError, native.SinkRouterError)):
                    call()
    assert launched == []
    for call in steps(**good):
        call()
    assert launched == ["route", "decode_attention_quant", "rope_append_route_kv", "decode_attention_quant"]


@pytest.mark.parametrize("quant", [False, True])
def test_shared_prefix_decoder_refuses_what_does_not_fit_before_it_launches(lib, launched, quant):
    B, Hq, Hkv, cap, L = 2, 8, 4, 20, 9
    dec = object.__new__(shared_prefix.SharedPrefixDecoder)
    dec.suffix = bare(native.Decoder, B, Hq, Hkv, L)
    dec.q = dec.workspace = dec.o_suffix = dec.lse_suffix = None
    if quant:
        c = native.QuantCache(B, Hkv, L, device="cpu")
        k, scales = c.k, c.scales
        caches = [native.QuantCache(1, Hkv, L, device="cpu").k, k.view(torch.int8), k.transpose(1, 2)]
    else:
        k, scales = half(B, Hkv, L, 128), None
        caches = [half(1, Hkv, L, 128), half(B, Hkv + 1, L, 128), k.float(), half(B, Hkv, L, 64), k.transpose(1, 2),
                  shifted(B, Hkv, L, 128), half(Hkv, L, 128)]
    rows = half(B, Hkv, 128)
    good = dict(q=half(B, Hq, 128), k_prefix=half(Hkv, cap, 128), v_prefix=half(Hkv, cap, 128), prefix_len=cap, k_cache=k,
                v_cache=k, k0=rows, v0=rows, seq_lens=torch.ones(B, dtype=torch.int32), n_splits=0)
    prefixes = [half(Hkv + 1, cap, 128), half(Hkv, cap, 64), half(Hkv, cap, 128).float(), half(cap, 128),
                half(cap, Hkv, 128).transpose(0, 1), shifted(Hkv, cap, 128)]
    bad = dict(q=[half(B + 1, Hq, 128), half(B, 16, 128), half(B, Hq, 128).float()], k_prefix=prefixes,
               v_prefix=prefixes + [half(Hkv, cap - 1, 128)], prefix_len=[-1, cap + 1], v_cache=caches,
               k0=[half(B + 1, Hkv, 128), half(B, Hkv + 1, 128)], v0=[half(1, Hkv, 128), rows.float()],
               seq_lens=[torch.ones(B + 1, dtype=torch.int32), torch.ones(B, dtype=torch.int64)],
               n_splits=[-2, 2000, native.SR_MAX_SPLITS + 1])
    bad["k_cache"] = [c for c in caches if c.dtype != torch.int8]

    def steps(q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, k0, v0, seq_lens, n_splits):
        yield lambda: dec.step(q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, k0, v0, seq_lens, 0.6, scales, n_splits)
        yield lambda: dec.append_step(q, rows, rows, None, None, k_prefix, v_prefix, prefix_len, k_cache, v_cache, k0, v0,
                                      seq_lens, 0.6, scales, n_splits)
    for name, values in bad.items():
        for v in values:
            for call in steps(**{**good, name: v}):
                with pytest.raises((ValueError, native.SinkRouterError)):
                    call()
    empty = half(Hkv, 0, 128)
    for call in steps(**{**good, "k_prefix": empty, "v_prefix": empty, "prefix_len": 0}):
        with pytest.raises(ValueError, match="prefix_len"):
            call()
    assert launched == []
    part = "decode_attention_quant_partial" if quant else "decode_attention_partial"
    for call in steps(**good):
        call()
    assert launched == ["route", part, "prefix_attention", "rope_append_route_kv", part, "prefix_attention"]


def test_step_graph_refuses_decoders_whose_step_takes_other_arguments(launched):
    """An 8-bit decoder's step would take the bf16 step's arguments one place off."""
    shape = half(1, 1, 128)
    for cls in (native.QuantDecoder, shared_prefix.SharedPrefixDecoder):
        with pytest.raises(TypeError, match=cls.__name__):
            native.StepGraph(object.__new__(cls), shape, shape, shape, shape, shape, shape, 0.6)
    assert launched == []
