"""The 8-bit KV cache without a GPU: argument checks of the C entry points before
any launch, the binding's refusals, and pins of the plain implementation that
the GPU tests compare against."""
import ctypes
import math

import pytest
import torch

import kv_plain as P
from oracle import dvssq_oracle as O


@pytest.fixture(scope="module")
def dv():
    import mixed_precision_weight_b200 as pkg
    return pkg.binding


def cache(dv, **kw):
    base = dict(k=256, v=256, k_scale=256, v_scale=256, table=256, n_pages=8, kv_heads=4,
                head_dim=128, batch=3, table_width=2)
    base.update(kw)
    return dv._KvCacheC(**base)


def append(dv, c, k=256, kts=512, khs=128, v=256, vts=512, vhs=128, T=3, start=256, cu=None):
    return dv.lib.dvssq_kv_append(None if c is None else ctypes.byref(c), k, kts, khs, v, vts, vhs, T,
                                  start, cu, None)


def read(dv, c, k=256, v=256, T=3, start=256, cu=None):
    return dv.lib.dvssq_kv_read(None if c is None else ctypes.byref(c), k, v, T, start, cu, None)


BAD_CACHES = [
    (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(kv_heads=0), 2), (dict(kv_heads=1025), 2),
    (dict(batch=0), 2), (dict(batch=4097), 2), (dict(n_pages=0), 2), (dict(table_width=0), 2),
    (dict(table_width=2 ** 18 + 1), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
    (dict(v_scale=None), 1), (dict(table=None), 1), (dict(k=264), 3), (dict(v=264), 3),
    (dict(k_scale=258), 3), (dict(v_scale=258), 3), (dict(table=258), 3),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_rejected(dv, kw, status):
    c = cache(dv, **{"table_width": 128, **kw})
    assert append(dv, c) == status
    assert read(dv, c) == status
    if "head_dim" not in kw and "kv_heads" not in kw and "batch" not in kw and "table_width" not in kw:
        assert attend(dv, c) == status


def test_append_and_read_argument_checks(dv):
    c = cache(dv)
    assert append(dv, None) == 1 and read(dv, None) == 1
    assert append(dv, c, T=0) == 0 and read(dv, c, T=0) == 0            # no-op, no device needed
    assert append(dv, c, T=-1) == 1 and append(dv, c, T=2 ** 30 + 1) == 1
    assert append(dv, c, T=4) == 1                                      # without cu: one row per sequence
    assert append(dv, c, k=None) == 1 and append(dv, c, v=None) == 1 and append(dv, c, start=None) == 1
    assert append(dv, c, kts=-8) == 1 and append(dv, c, vhs=-8) == 1
    assert append(dv, c, kts=516) == 3 and append(dv, c, khs=4) == 3 and append(dv, c, vts=2) == 3
    assert append(dv, c, k=264) == 3 and append(dv, c, v=264) == 3
    assert append(dv, c, start=258) == 3 and append(dv, c, T=7, cu=262) == 3
    assert read(dv, c, k=None) == 1 and read(dv, c, v=None) == 1
    assert read(dv, c, k=264) == 3 and read(dv, c, v=264) == 3 and read(dv, c, start=258) == 3


def attend(dv, c, shape=None, q=256, qbs=2048, qhs=128, lens=256, out=256, yd=0, ws=256, wsb=1 << 40,
           prefix=None, plen=0, entry="q8"):
    sh = dv.AttnShape(3, 16, 4, 128, 8192, 1.1, 12.0) if shape is None else shape
    shp = None if sh is False else ctypes.byref(sh)
    cp = None if c is None else ctypes.byref(c)
    if entry == "q8":
        return dv.lib.dvssq_bss_attention_q8(shp, cp, q, qbs, qhs, lens, out, yd, ws, wsb, None)
    return dv.lib.dvssq_bss_attention_prefix(shp, cp, prefix, plen, q, qbs, qhs, lens, out, yd, ws, wsb, None)


def test_attention_argument_checks(dv):
    n = ctypes.c_size_t(0)
    tiny = dv.AttnShape(3, 16, 4, 128, 128, 1.1, 12.0)
    assert dv.lib.dvssq_bss_attention_q8_workspace_size(ctypes.byref(tiny), ctypes.byref(n)) == 0
    assert n.value == 0                                                  # one launch, no partial sums
    c = cache(dv, table_width=128)
    good = dv.AttnShape(3, 16, 4, 128, 8192, 1.1, 12.0)
    assert dv.lib.dvssq_bss_attention_q8_workspace_size(ctypes.byref(good), ctypes.byref(n)) == 0
    need = n.value
    assert need > 0
    assert dv.lib.dvssq_bss_attention_q8_workspace_size(ctypes.byref(good), None) == 1
    assert dv.lib.dvssq_bss_attention_q8_workspace_size(None, ctypes.byref(n)) == 1
    assert dv.lib.dvssq_bss_attention_prefix_workspace_size(ctypes.byref(good), 5000, ctypes.byref(n)) == 0
    assert n.value > need
    assert dv.lib.dvssq_bss_attention_prefix_workspace_size(ctypes.byref(good), -1, ctypes.byref(n)) == 1
    assert dv.lib.dvssq_bss_attention_prefix_workspace_size(ctypes.byref(good), 2 ** 24 + 1, ctypes.byref(n)) == 2
    A = dv.AttnShape
    for sh, status in ((A(0, 16, 4, 128, 128, 1.1, 12.0), 2), (A(4097, 16, 4, 128, 128, 1.1, 12.0), 2),
                       (A(3, 15, 4, 128, 128, 1.1, 12.0), 2), (A(3, 68, 4, 128, 128, 1.1, 12.0), 2),
                       (A(3, 0, 4, 128, 128, 1.1, 12.0), 2), (A(3, 16, 0, 128, 128, 1.1, 12.0), 2),
                       (A(3, 16, 4, 96, 128, 1.1, 12.0), 2), (A(3, 16, 4, 128, 0, 1.1, 12.0), 2),
                       (A(3, 16, 4, 128, 2 ** 24 + 1, 1.1, 12.0), 2), (A(4096, 16, 4, 128, 2 ** 23, 1.1, 12.0), 2),
                       (A(3, 16, 4, 128, 128, 0.0, 12.0), 1),
                       (A(3, 16, 4, 128, 128, math.nan, 12.0), 1), (A(3, 16, 4, 128, 128, math.inf, 12.0), 1),
                       (A(3, 16, 4, 128, 128, 1.1, math.nan), 1),
                       # not the cache's own shape, or longer than its table
                       (A(2, 16, 4, 128, 128, 1.1, 12.0), 1), (A(3, 16, 2, 128, 128, 1.1, 12.0), 1),
                       (A(3, 16, 4, 256, 128, 1.1, 12.0), 1), (A(3, 16, 4, 128, 8193, 1.1, 12.0), 1)):
        assert attend(dv, c, sh) == status, tuple(getattr(sh, f) for f, _ in sh._fields_)
    for entry in ("q8", "prefix"):
        call = lambda cc=c, **kw: attend(dv, cc, entry=entry, **kw)  # noqa: E731
        assert call(shape=False) == 1 and call(cc=None) == 1
        assert call(q=None) == 1 and call(lens=None) == 1 and call(out=None) == 1 and call(ws=None) == 1
        assert call(yd=2) == 1 and call(qbs=-8) == 1
        assert call(qbs=2044) == 3 and call(qhs=100) == 3
        assert call(q=264) == 3 and call(lens=258) == 3 and call(out=264) == 3 and call(ws=272) == 3
        assert call(wsb=need - 256) == 4
    assert attend(dv, c, entry="prefix", plen=-1, prefix=256) == 1
    assert attend(dv, c, entry="prefix", plen=100, prefix=None) == 1
    assert attend(dv, c, entry="prefix", plen=100, prefix=262) == 3
    assert attend(dv, c, entry="prefix", plen=5000, prefix=256, wsb=need) == 4


def test_workspace_is_bounded_by_the_context(dv):
    # fp32 logits (8 B of slack per key and head) dominate a long context's workspace
    sh = dv.AttnShape(4, 16, 4, 256, 32768, 1.1, 12.0)
    assert dv.dvssq_bss_attention_q8_workspace_size(sh) <= 4 * 16 * 32768 * 8 + (64 << 20)


def test_binding_refusals_without_a_gpu(dv):
    table = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):                        # a host pool never reaches a kernel
        dv.KvCache.zeros(4, 2, 128, table)
    k = torch.zeros((4, 2, 64, 128), dtype=torch.int8)
    s = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dv.KvCache(k.float(), k.transpose(2, 3).contiguous(), s, s, table)
    with pytest.raises(ValueError):
        dv.KvCache(k[0], k, s, s, table)
    with pytest.raises(TypeError):                                       # indices are int32
        dv._indices(table.long(), "start", 6, -1)
    with pytest.raises(ValueError):
        dv._indices(table, "start", 5, -1)
    with pytest.raises(ValueError, match="cuda:0"):                      # a host tensor beside a CUDA cache
        dv._indices(table, "start", 6, 0)
    rows = torch.zeros((5, 2, 128), dtype=torch.bfloat16)
    assert dv._rows(rows, "k", (5, 2, 128), -1)[1:] == (256, 128)
    fused = torch.zeros((5, 8, 128), dtype=torch.bfloat16)[:, 4:6]
    assert dv._rows(fused, "k", (5, 2, 128), -1)[1:] == (1024, 128)
    with pytest.raises(TypeError):
        dv._rows(rows.float(), "k", (5, 2, 128), -1)
    with pytest.raises(ValueError):
        dv._rows(rows, "k", (5, 2, 64), -1)
    with pytest.raises(ValueError):
        dv._rows(torch.zeros((5, 128, 2), dtype=torch.bfloat16).transpose(1, 2), "k", (5, 2, 128), -1)


# ----------------------------------------------- pins of the plain implementation
def test_plain_hold_is_the_int8_tier():
    x = P.queries(5, 3, 64, seed=1)
    c, s = P.hold(x)
    f = O.torch_bf16_to_f64(x.reshape(-1, 64))
    q8, s8 = O.quantize_int8(f, range(64))
    assert (c.reshape(-1, 64).numpy() == q8).all()
    assert (O.torch_bf16_to_f64(s.reshape(-1)) == s8).all()


def test_plain_attention_is_the_oracle_on_the_held_values():
    q = P.queries(2, 8, 64, seed=2)
    lens = [150, 150]
    pool, table, _ = P.filled(2, 4, 64, lens, seed=3, bind=(q, 15.0))
    kv = [P.keys_values(pool, table[b], 150) for b in range(2)]
    ref = O.bss_attention(O.torch_bf16_to_f64(q), torch.stack([x[0] for x in kv]).numpy(),
                          torch.stack([x[1] for x in kv]).numpy())
    got = P.attention(q, pool, table, lens)
    assert torch.allclose(got, torch.from_numpy(ref), rtol=1e-12, atol=1e-13)


def test_plain_prefix_is_attention_over_the_concatenation():
    q = P.queries(1, 4, 64, seed=4)
    pool, table, ptable = P.filled(1, 2, 64, [70], seed=5, prefix=100)
    a = P.attention(q, pool, table, [70], ptable=ptable, prefix=100)
    pk, pv = P.keys_values(pool, ptable, 100)
    k, v = P.keys_values(pool, table[0], 70)
    ref = O.bss_attention(O.torch_bf16_to_f64(q), torch.cat([pk, k], 1)[None].numpy(),
                          torch.cat([pv, v], 1)[None].numpy())
    assert torch.allclose(a, torch.from_numpy(ref), rtol=1e-12, atol=1e-13)


def test_plain_append_then_read_round_trip():
    g = torch.Generator().manual_seed(6)
    pool, table, _ = P.filled(2, 2, 64, [100, 130], seed=7)
    k = torch.randn((9, 2, 64), generator=g).to(torch.bfloat16)
    v = torch.randn((9, 2, 64), generator=g).to(torch.bfloat16)
    start, cu = [61, 10], [0, 5, 9]
    P.append(pool, table, k, v, start, cu)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    P.read(pool, table, start, cu, ko, vo)
    # half a step of the row's scale, half a BF16 step of the scale (up to 127 / 256 of a
    # step at the largest code), then half a BF16 step of the value
    for a, b in ((k, ko), (v, vo)):
        step = a.double().abs().amax(-1, keepdim=True) / 127
        assert ((a.double() - b.double()).abs() <= step * (0.5 + 0.5) + b.double().abs() * 2 ** -8).all()
