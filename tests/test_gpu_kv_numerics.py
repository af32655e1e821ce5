"""KV-BSS attention over the 8-bit cache where the numbers are far from ordinary: large
logits, haze thresholds below the logits' own rounding, equal largest keys before and
behind a prefix's end.  Every form of the kernels against the plain 64-bit implementation
(kv_plain.py).

Tolerances, relative L2 error of one head's output.  A row whose largest logit leads the
others by more than `clear` has one weight, so that the output is that key's value: nothing
is off but roundings of the weight itself (two BF16 limbs 2^-17, FP16 2^-11 = 4.9e-4) and of
FP32 products.  `clear` is the threshold or, where there is none or a wide one, 20 (every
other weight then is below 2e-9), plus the rounding of both logits: FP32 operations on
partial sums of up to 256 products, at most 2^-19 of the larger logit.
"""
import math

import pytest
import torch

import kv_plain as P
from test_gpu_kv_cache import DECODE, PREFIX, check, i32, to_gpu, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dv():
    import mixed_precision_weight_b200 as pkg
    return pkg.binding


@pytest.fixture(autouse=True)
def no_device_error(dv):
    dv.dvssq_device_error(clear=True)
    yield
    assert dv.dvssq_device_error(clear=True) == 0


def leads(q, pool, table, lens, ptable, prefix, tau):
    """The largest logit's magnitude and its lead over the next key's, [B][Hq] each (fp64)."""
    B, Hq, d = q.shape
    H = pool["k"].shape[1]
    top, lead = torch.zeros(B, Hq, dtype=torch.float64), torch.full((B, Hq), math.inf, dtype=torch.float64)
    for b in range(B):
        k, _ = P.keys_values(pool, table[b], int(lens[b]))
        if prefix:
            k = torch.cat([P.keys_values(pool, ptable, prefix)[0], k], 1)
        s = torch.einsum("hgd,hld->hgl", q[b].double().reshape(H, -1, d), k).reshape(Hq, -1) * (tau / math.sqrt(d))
        x = s.topk(min(2, s.shape[1]), dim=-1).values
        top[b] = s.abs().amax(-1)
        if x.shape[1] == 2:
            lead[b] = x[:, 0] - x[:, 1]
    return top, lead


def check_winners(got, ref, top, lead, haze, bound):
    clear = (haze if 0 < haze < 20 else 20.0) + top * 2.0 ** -19
    rows = lead > clear
    assert rows.double().mean() > 0.9                       # the inputs hold what the test is about
    check(got[rows.to(got.device)][None], ref[rows][None], bound)


# (query heads, KV heads, d, own lengths, prefix): enough visits that the prefix is read once
READ_ONCE = [(8, 8, 64, [17, 0] * 20, 897), (16, 2, 128, [0, 70, 1] * 12, 3800), (16, 1, 128, [9] * 60, 2700),
             (16, 4, 256, [1, 300] * 9, 3700)]
# tau, haze: logits near 100, 1e4, 1e6, 1e10 and 1e20
SHARP = [(30.0, 1e-6), (30.0, 1e-30), (3000.0, 1e-3), (3000.0, 12.0), (1e6, 12.0), (1e10, 12.0), (1e10, 0.0), (1e20, 12.0)]


@pytest.mark.parametrize("Hq,H,d,lens,prefix", READ_ONCE)
def test_prefix_read_once_keeps_its_largest_key(dv, Hq, H, d, lens, prefix):
    B = len(lens)
    assert B * H * -(-prefix // 64) > (4096 if Hq // H <= 8 else 2400)
    q = P.queries(B, Hq, d, seed=prefix)
    pool, table, ptable = P.filled(B, H, d, lens, seed=prefix + 1, prefix=prefix)
    c, lg, pg, qg = to_gpu(dv, pool, table), i32(lens), ptable.cuda(), q.cuda()
    for tau, haze in SHARP:
        out = dv.dvssq_bss_attention_prefix(qg, c, lg, pg, prefix, tau=tau, haze=haze)
        assert torch.isfinite(out).all(), (tau, haze)
        ref = P.attention(q, pool, table, lens, tau=tau, haze=haze, ptable=ptable, prefix=prefix)
        check_winners(out, ref, *leads(q, pool, table, lens, ptable, prefix, tau), haze, PREFIX)


@pytest.mark.parametrize("Hq,H,d", [(8, 8, 64), (16, 2, 128), (16, 1, 128), (16, 4, 256)])
def test_decode_keeps_its_largest_key(dv, Hq, H, d):
    lens = [1300, 64, 1, 1025, 700]
    q = P.queries(5, Hq, d, seed=d)
    pool, table, _ = P.filled(5, H, d, lens, seed=d + 1)
    for tau, haze in SHARP:
        ref = P.attention(q, pool, table, lens, tau=tau, haze=haze)
        top = leads(q, pool, table, lens, None, 0, tau)
        for width in (0, 33, 129):
            out = dv.dvssq_bss_attention_q8(q.cuda(), widened(dv, pool, table, width), i32(lens), tau=tau, haze=haze)
            # the query's rounding moves a logit by at most 2^-15 max|q| sum|k| tau / sqrt(d), with
            # max|q| below 4 and |k| near 1 2e-3 tau of logits of 3.3 tau: less than 2^-10 for two keys
            check_winners(out, ref, top[0], top[1] - top[0] * 2.0 ** -10, haze, DECODE)


@pytest.mark.parametrize("tau", [1.1, 1e3, 3e5, 1e7, 1e12])
def test_equal_largest_keys_in_prefix_and_own_part(dv, tau):
    """One key row stands in the prefix and among the own keys, with different values, and leads all
    others: both weigh one half.  The query's values are +-1 and +-2, so that q . k is exact in
    every form and both logits are the same roundings of the same number."""
    lens, prefix, d = [5, 70, 130] * 12, 3800, 128
    B, Hq, H = len(lens), 16, 2
    g = torch.Generator().manual_seed(7)
    q = (torch.randint(1, 3, (B, Hq, d), generator=g) * (2 * torch.randint(0, 2, (B, Hq, d), generator=g) - 1)).to(torch.bfloat16)
    q[:] = q[:1, ::8].repeat_interleave(8, 1)               # the planted key leads for every head and sequence
    pool, table, ptable = P.filled(B, H, d, lens, seed=8, prefix=prefix, std=0.25)
    kc, ks = P.hold(2.0 * q[0, ::8])                        # [H][d], logits near 2 tau 300 / sqrt(d)
    places = [(int(ptable[1700 // 64]), 1700 % 64)] + [(int(table[b, 0]), 3) for b in range(B)]
    for page, slot in places:
        pool["k"][page, :, slot], pool["ks"][page, :, slot] = kc, ks
    c = to_gpu(dv, pool, table)
    ref = P.attention(q, pool, table, lens, tau=tau, ptable=ptable, prefix=prefix)
    out = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), ptable.cuda(), prefix, tau=tau)
    check(out, ref, PREFIX)


@pytest.mark.parametrize("up", [111, -111, 60, -60])
@pytest.mark.parametrize("Hq,H,d", [(8, 8, 64), (16, 2, 128), (16, 1, 128), (16, 4, 256)])
def test_ordinary_logits_of_huge_and_tiny_factors(dv, Hq, H, d, up):
    """Keys times 2^up and queries times 2^-up: the logits are those of neither, bit for bit in exact
    arithmetic, so that the bounds are the ordinary ones."""
    lens = [1300, 64, 1, 0, 700, 130, 65]
    q = P.queries(7, Hq, d, seed=d)
    prefix = 64 * ((4096 if Hq // H <= 8 else 2400) // (7 * H) + 1) - 27
    pool, table, ptable = P.filled(7, H, d, lens, seed=d + 1, prefix=prefix)
    ref = P.attention(q, pool, table, lens)
    both = P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix)
    pool["ks"] = (pool["ks"].float() * 2.0 ** up).to(torch.bfloat16)
    assert not pool["ks"].isinf().any()
    qg = (q.float() * 2.0 ** -up).to(torch.bfloat16).cuda()
    assert torch.equal(qg.cpu().double() * 2.0 ** up, q.double())           # no bit was lost
    for width in (0, 33, 130):
        check(dv.dvssq_bss_attention_q8(qg, widened(dv, pool, table, width), i32(lens)), ref, DECODE)
    for width in (0, 17):
        c = widened(dv, pool, table, width)
        check(dv.dvssq_bss_attention_prefix(qg, c, i32(lens), ptable.cuda(), prefix), both, PREFIX)
    c = widened(dv, pool, table, 0)
    few = P.attention(q, pool | {"ks": (pool["ks"].float() * 2.0 ** -up).to(torch.bfloat16)}, table, lens,
                      ptable=ptable, prefix=100)
    check(dv.dvssq_bss_attention_prefix(qg, c, i32(lens), ptable[:2].cuda(), 100), few, DECODE)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_extreme_rows_read_back_exactly(dv, d):
    """Rows from the smallest subnormal to the largest BF16 value: every value read back is the exact
    product of its code and scale, rounded once (subnormal results among them)."""
    g = torch.Generator().manual_seed(d)
    exps = [-133, -130, -127, -126, -125, -120, -110, -95, -90, -60, 0, 60, 100, 120, 124, 125]
    x = torch.stack([(torch.randn(1, d, generator=g) * 2.0 ** (e / 2)).to(torch.bfloat16).float() * 2.0 ** (e - e / 2)
                     for e in exps]).clamp(-3.3895313892515355e38, 3.3895313892515355e38).to(torch.bfloat16)
    x[-1, 0, :2] = torch.tensor([3.3895313892515355e38, -3.3895313892515355e38]).to(torch.bfloat16)
    T = len(exps)
    pool, table, _ = P.filled(1, 1, d, [T], seed=d)
    pool["ks"].nan_to_num_(0.0)
    pool["vs"].nan_to_num_(0.0)
    c = to_gpu(dv, pool, table)
    P.append(pool, table, x, x.flip(0), [0], [0, T])
    dv.dvssq_kv_append(c, x.cuda(), x.flip(0).contiguous().cuda(), i32([0]), i32([0, T]))
    assert torch.equal(c.k_scale.cpu(), pool["ks"]) and torch.equal(c.v_scale.cpu(), pool["vs"])
    assert torch.equal(c.k.cpu(), pool["k"]) and torch.equal(c.v.cpu(), pool["v"])
    ko, vo = torch.zeros_like(x), torch.zeros_like(x)
    P.read(pool, table, [0], [0, T], ko, vo)
    # (the largest value's scale is rounded up: 127 of its steps are past BF16's range)
    assert torch.isfinite(ko[:-1].float()).all() and (ko != 0).any(-1).sum() >= T - 5
    k, v = dv.dvssq_kv_read(c, i32([0]), i32([0, T]), T)
    assert torch.equal(k.cpu(), ko) and torch.equal(v.cpu(), vo)
