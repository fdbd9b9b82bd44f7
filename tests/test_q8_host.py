"""The 8-bit cache's entry points refuse bad arguments on the host, and the
64-bit reference of their tests is right (CPU only: no CUDA call is reached)."""
import ctypes
import math

import pytest
import torch

import long_context_indexer_b200 as lci
from long_context_indexer_b200.build import build

from . import q8_reference as ref

INVALID, UNSUPPORTED = 1, 2
FAKE = ctypes.c_void_p(0x7F0000000000)
ODD = ctypes.c_void_p(0x7F0000000008)


@pytest.fixture(scope="module")
def lib():
    build()
    return lci.load_library()


@pytest.fixture(scope="module")
def tables(lib):
    made = {}
    for name, (nb, P, bs, H, hd, dt) in dict(
            q8=(4, 8, 64, 2, 128, 2), bf16=(4, 8, 64, 2, 128, 1), odd=(4, 8, 64, 2, 48, 2),
            wide=(4, 8, 64, 2, 288, 2), long=(1 << 15, 8, 64, 2, 128, 2),
            huge=(1 << 25, 8, 64, 2, 128, 2)).items():
        h = ctypes.c_void_p()
        assert lib.lci_create_block_table(FAKE, 2, nb, P, bs, H, hd, dt, ctypes.byref(h)) == 0
        made[name] = h
    yield made
    for h in made.values():
        lib.lci_destroy_block_table(h)


def test_other_attention_refuses_an_e4m3_table(lib, tables):
    assert lib.lci_sparse_attn(FAKE, 2, 1, 16, FAKE, FAKE, tables["q8"], FAKE, 4, FAKE, FAKE, 0.0, 0,
                               FAKE, None, 0, None) == UNSUPPORTED
    assert lib.lci_sparse_attn_partial(FAKE, 2, 1, 16, FAKE, FAKE, tables["q8"], FAKE, 4, FAKE, FAKE,
                                       0.0, 0, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.lci_sparse_attn_pipelined(FAKE, 2, 1, 16, FAKE, FAKE, tables["q8"], FAKE, 4, FAKE,
                                         FAKE, 0.0, FAKE, FAKE, None) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.lci_sparse_decode_workspace_size(2, 1, 8, 128, 4, 16, tables["q8"],
                                                ctypes.byref(n)) != 0
    for fn in (lib.lci_sparse_decode, lib.lci_sparse_decode_persistent):
        for dtype in (0, 1, 2):
            assert fn(FAKE, FAKE, dtype, 2, 1, 8, 128, 4, FAKE, FAKE, 4, FAKE, 16, FAKE, FAKE,
                      tables["q8"], 0.0, FAKE, FAKE, FAKE, 1 << 30, None) in (INVALID, UNSUPPORTED)
    h = ctypes.c_void_p()
    assert lib.lci_create_block_table(FAKE, 2, 4, 8, 64, 2, 128, 3, ctypes.byref(h)) == INVALID


def test_kv_append_q8_refusals(lib, tables):
    def call(**kw):
        a = dict(k=FAKE, v=FAKE, dtype=1, B=2, T=1, start=FAKE, count=None, t=tables["q8"], kp=FAKE,
                 vp=FAKE, ks=FAKE, vs=FAKE)
        a.update(kw)
        return lib.lci_kv_append_q8(*a.values(), None)
    for name in ("k", "v", "start", "kp", "vp", "ks", "vs", "t"):
        assert call(**{name: None}) == INVALID, name
    assert call(B=0) == INVALID and call(B=3) == INVALID and call(T=0) == INVALID
    assert call(dtype=2) == INVALID and call(dtype=9) == INVALID
    assert call(t=tables["bf16"]) == INVALID
    assert call(kp=ODD) == INVALID and call(vp=ODD) == INVALID


def test_sparse_attn_q8_refusals(lib, tables):
    class Opt(ctypes.Structure):
        _fields_ = [("cap", ctypes.c_float), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                    ("c", ctypes.c_void_p)]

    def call(**kw):
        a = dict(q=FAKE, dtype=1, B=2, S=1, Hq=16, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE,
                 t=tables["q8"], ids=FAKE, topk=4, ctx=FAKE, q0=FAKE, scale=0.0, opt=None, phase=0,
                 out=FAKE, lse=None, mass=None)
        a.update(kw)
        return lib.lci_sparse_attn_q8(*a.values(), None)
    for name in ("q", "kp", "vp", "ks", "vs", "t", "ids", "ctx", "q0", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(S=0) == INVALID and call(Hq=15) == INVALID and call(topk=0) == INVALID
    assert call(B=3) == INVALID and call(dtype=2) == INVALID and call(phase=3) == INVALID
    assert call(t=tables["bf16"]) == INVALID
    assert call(q=ODD) == INVALID and call(out=ODD) == INVALID and call(vp=ODD) == INVALID
    assert call(scale=float("inf")) == INVALID
    for cap in (-1.0, float("nan"), float("inf")):
        assert call(opt=ctypes.byref(Opt(cap, None, None, None))) == INVALID
    assert call(topk=257) == UNSUPPORTED
    assert call(t=tables["odd"]) == UNSUPPORTED and call(t=tables["wide"]) == UNSUPPORTED
    assert call(t=tables["huge"]) == UNSUPPORTED


def test_block_weight_update_refusals(lib):
    def call(**kw):
        a = dict(ids=FAKE, mass=FAKE, B=2, S=1, H=1, topk=4, NB=16, decay=1.0, w=FAKE)
        a.update(kw)
        return lib.lci_block_weight_update(*a.values(), None)
    for name in ("ids", "mass", "w"):
        assert call(**{name: None}) == INVALID
    for name in ("B", "S", "H", "topk", "NB"):
        assert call(**{name: 0}) == INVALID
    for decay in (-0.5, float("nan"), float("inf")):
        assert call(decay=decay) == INVALID
    assert call(topk=257) == UNSUPPORTED and call(NB=16385) == UNSUPPORTED


def test_cache_evict_refusals(lib, tables):
    def call(**kw):
        a = dict(t=tables["q8"], B=2, ctx=FAKE, w=FAKE, budget=3, sink=1, recent=1, to=FAKE, co=FAKE,
                 wo=FAKE, kept=None, freed=None)
        a.update(kw)
        return lib.lci_cache_evict(*a.values(), None)
    for name in ("t", "ctx", "w", "to", "co", "wo"):
        assert call(**{name: None}) == INVALID
    assert call(B=0) == INVALID and call(B=3) == INVALID
    assert call(sink=-1) == INVALID and call(recent=0) == INVALID
    assert call(sink=2, recent=2) == INVALID and call(budget=0) == INVALID
    assert call(t=tables["long"]) == UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        lci.block_weight_update(torch.zeros(1, 4), torch.zeros(1, 1, 2, dtype=torch.int32),
                                torch.zeros(1, 1, 1, 2))


# ---------------------------------------------------------------- the reference

def test_reference_rounds_to_e4m3_like_torch():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(4000, generator=g) * s for s in (1e-3, 0.01, 1.0, 100.0)]).clamp(-448, 448)
    mid = ((ref.E4M3[1:] + ref.E4M3[:-1]) / 2).float()  # ties
    x = torch.cat([x, mid, -mid, ref.E4M3.float(), torch.zeros(1)])
    assert torch.equal(ref.e4m3_round(x.double()).float(), x.to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("amax", [448.0, 448.0001, 1.0, 3.5, 1.75, 1e-30, 0.0, 3e38])
def test_reference_scale_is_the_smallest_that_fits(amax):
    s = ref.needed_scale(amax)
    assert math.log2(s) == int(math.log2(s)) and s >= 2.0 ** -60 and 448 * s >= amax
    assert s == 2.0 ** -60 or 448 * s / 2 < amax


def test_reference_attention_is_dense_attention():
    g = torch.Generator().manual_seed(1)
    bs, H, hd, n = 4, 2, 8, 11
    k = torch.randn(5, H, bs, hd, generator=g).to(torch.float8_e4m3fn)
    v = torch.randn(5, H, bs, hd, generator=g).to(torch.float8_e4m3fn)
    ks, vs = torch.rand(5, H, generator=g) + 0.5, torch.rand(5, H, generator=g) + 0.5
    table = torch.tensor([[3, 0, 4]], dtype=torch.int32)
    q = torch.randn(1, n, 4, hd, generator=g)
    ids = torch.tensor([2, 0, 1], dtype=torch.int32).repeat(1, n, 1)
    out, lse, mass, _ = ref.attend(q.double(), k.double(), v.double(), ks, vs, table, bs, ids,
                                   torch.tensor([n]), torch.tensor([0]))
    K = (k.double() * ks.double()[:, :, None, None])[table[0].long()].transpose(0, 1).reshape(H, -1, hd)[:, :n]
    V = (v.double() * vs.double()[:, :, None, None])[table[0].long()].transpose(0, 1).reshape(H, -1, hd)[:, :n]
    want = torch.nn.functional.scaled_dot_product_attention(
        q[0].transpose(0, 1).double(), K.repeat_interleave(2, 0), V.repeat_interleave(2, 0), is_causal=True)
    assert torch.allclose(out[0].transpose(0, 1), want, atol=1e-12)
    assert torch.allclose(mass.sum(-1), torch.full((1, n, H), 2.0, dtype=torch.float64))


# entry: its arguments without the stream, and changes by position that are refused
PREPARED_CASES = {
    "lci_kv_append_q8": (
        lambda t: [FAKE, FAKE, 1, 2, 1, FAKE, None, t, FAKE, FAKE, FAKE, FAKE],
        {0: None, 1: None, 2: 7, 3: 3, 4: 0, 5: None, 7: None, 8: ODD, 9: ODD, 10: None, 11: None}),
    "lci_sparse_attn_q8": (
        lambda t: [FAKE, 1, 2, 1, 16, FAKE, FAKE, FAKE, FAKE, t, FAKE, 4, FAKE, FAKE, 0.0, None, 0,
                   FAKE, None, None],
        {0: ODD, 1: 7, 2: 3, 3: -5, 4: 15, 5: ODD, 6: ODD, 7: None, 8: None, 9: None, 10: None,
         11: 257, 12: None, 13: None, 14: math.inf, 16: 9, 17: None}),
    "lci_block_weight_update": (
        lambda t: [FAKE, FAKE, 2, 1, 2, 4, 8, 0.5, FAKE],
        {0: None, 1: None, 2: 65536, 3: 0, 4: -1, 5: 257, 6: 16385, 7: -0.5, 8: None}),
    "lci_cache_evict": (
        lambda t: [t, 2, FAKE, FAKE, 4, 1, 1, FAKE, FAKE, FAKE, None, None],
        {0: None, 1: 3, 2: None, 3: None, 4: 1, 5: -1, 6: 0, 7: None, 8: None, 9: None}),
}


@pytest.mark.parametrize("name", PREPARED_CASES)
def test_prepared_call_passes_each_argument_in_its_place(lib, tables, name):
    """A refused argument is refused alike, and with the same words, by both forms of the call."""
    from long_context_indexer_b200.lci import _PREPARED, _pack_args
    base, changes = PREPARED_CASES[name]
    direct = getattr(lib, name)
    messages = set()
    for at, bad in changes.items():
        args = base(tables["q8"])
        args[at] = bad
        rc = direct(*args, None)
        words = lib.lci_last_error()
        assert rc in (INVALID, UNSUPPORTED), (at, bad)
        packed = _pack_args(name, tuple(args))
        assert lib.lci_call_prepared(_PREPARED[name], ctypes.addressof(packed), None) == rc
        assert lib.lci_last_error() == words
        messages.add(words)
    assert len(messages) >= 3


def test_prepared_call_refusals(lib):
    from long_context_indexer_b200.lci import _pack_args
    packed = _pack_args("lci_cache_evict", tuple(PREPARED_CASES["lci_cache_evict"][0](None)))
    assert lib.lci_call_prepared(3, None, None) == INVALID
    assert lib.lci_call_prepared(-1, ctypes.addressof(packed), None) == INVALID
    assert lib.lci_call_prepared(4, ctypes.addressof(packed), None) == INVALID
    with pytest.raises(ValueError):
        _pack_args("lci_cache_evict", (None, 2, FAKE, FAKE, 1 << 31, 1, 1, FAKE, FAKE, FAKE, None, None))
    with pytest.raises(TypeError):
        _pack_args("lci_cache_evict", (None, 2))


def _table(lib):
    t = object.__new__(lci.BlockTable)  # a handle over no device memory
    t._handle, t._lib = ctypes.c_void_p(), lib
    assert lib.lci_create_block_table(FAKE, 2, 4, 8, 64, 2, 128, 2, ctypes.byref(t._handle)) == 0
    return t


class _Stream:
    cuda_stream = None


def test_calls_prepared_over_a_closed_table_are_refused(lib, monkeypatch):
    import long_context_indexer_b200.lci as binding
    made = []
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    t = _table(lib)
    args = (t.handle, 2, FAKE, FAKE, 4, 1, 1, FAKE, FAKE, FAKE, None, None)
    call = binding.PreparedCall("lci_cache_evict", args, None, torch.device("cuda", 0), (t,))
    call._fn = lambda *a: made.append(a) or 0
    call(_Stream)
    assert len(made) == 1
    t.close()
    with pytest.raises(ValueError, match="closed"):
        call(_Stream)
    step = object.__new__(lci.SparseDecodeStep)
    step._name, step._keep, step._args = "lci_sparse_decode", (_table(lib),), (None,)
    step._fn = lambda *a: made.append(a) or 0
    step._keep[-1].register(step)  # as its constructor, which needs a GPU's tensors, does
    step()
    assert len(made) == 2
    step._keep[-1].close()
    with pytest.raises(ValueError, match="closed"):
        step()
    assert len(made) == 2


def test_caps_outside_the_range_are_refused(lib, tables):
    """A cap whose reciprocal is infinite would turn scores of zero into NaN."""
    class Opt(ctypes.Structure):
        _fields_ = [("cap", ctypes.c_float), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("c", ctypes.c_void_p)]
    for cap in (1e-40, 2.0 ** -101, 2.0 ** 101, 3e38, -0.5):
        opt = Opt(cap, None, None, None)
        assert lib.lci_sparse_attn_q8(FAKE, 1, 2, 1, 16, FAKE, FAKE, FAKE, FAKE, tables["q8"], FAKE, 4, FAKE, FAKE, 0.0,
                                      ctypes.byref(opt), 0, FAKE, None, None, None) == INVALID, cap
        assert b"cap" in lib.lci_last_error()


@pytest.mark.parametrize("names,limit,bound", [("C0 C1 C2 C3 C4", 0.625, 1e-8), ("T0 T1 T2", 0.25, 4e-9)])
def test_tanh_polynomials_are_the_fit(names, limit, bound):
    """The coefficients are a least squares fit of the relative error of
    u + u^3 (c0 + c1 u^2 + ...) at Chebyshev nodes of u^2 in [0, limit^2]."""
    import os
    import re

    import numpy as np
    src = open(os.path.join(os.path.dirname(lci.__file__), "csrc", "attn_q8_simt.cuh")).read()
    have = np.array([float(re.search(rf"kTanh{n} = (-?[0-9.]+)f", src).group(1)) for n in names.split()])
    k = np.arange(400)
    v = limit ** 2 * (0.5 - 0.5 * np.cos((2 * k + 1) * np.pi / 800))
    u = np.sqrt(v)
    weight = v * u / np.tanh(u)
    fit = np.linalg.lstsq(np.vander(v, len(have), increasing=True) * weight[:, None],
                          (np.tanh(u) / u - 1) / v * weight, rcond=None)[0]
    assert np.allclose(have, fit, rtol=1e-6, atol=0)
    u = np.linspace(1e-4, limit, 100001)
    poly = u + u ** 3 * sum(c * u ** (2 * i) for i, c in enumerate(have))
    assert np.abs(poly / np.tanh(u) - 1).max() <= bound


def test_weight_parts_add_up():
    """The tile schedule's three 8-bit parts of a weight, for every f16 that a
    weight can be: within 2^-9 of it, or 2^-17 where it is below 2^-8."""
    bits = torch.arange(1, int(torch.tensor(2.0 ** 15.75, dtype=torch.float16).view(torch.int16)) + 1, dtype=torch.int32)
    w = bits.to(torch.int16).view(torch.float16)

    def upper(x):  # the e5m2 number in the upper byte
        return (x.view(torch.int16) & -256).view(torch.float16)
    p0 = upper(w)
    p1 = upper(w - p0)
    p2 = upper((w - p0 - p1).view(torch.int16).add(0x80).view(torch.float16))
    for p in (p0, p1, p2):
        assert torch.equal(p.to(torch.float8_e5m2).to(torch.float16), p)
    off = (p0.double() + p1.double() + p2.double() - w.double()).abs()
    large = w >= 2.0 ** -8
    assert (off[large] <= w.double()[large] * 2.0 ** -9).all() and (off[~large] <= 2.0 ** -17).all()
