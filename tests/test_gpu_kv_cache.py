"""The 8-bit KV cache on the GPU against the plain 64-bit implementation
(kv_plain.py): quantising on write, reading back, KV-BSS decode attention over
the cache and over a shared prefix, and a decode loop of them together.

Write and read are exact: the scale and every code are decided by exact
quotients, and a value c s is one rounding of an exact product.

Attention tolerances, on random rows (relative L2 error of one head's output):
a weight's relative error is its logit's absolute error plus its own rounding,
and independent weight errors of rms e give an output error of about e.
- Decode: queries as 16-bit integers of a power-of-two step 2^-14 of the
  head's largest magnitude: exact for the BF16 values of the top 8 binades, at
  most 2^-15 of the largest for the others (about 2 % of them).  With d = 256,
  max|q| near 3.5 and |k| near 1 (4 for planted keys) the logit error is about
  2e-5 at most; weights in two BF16 limbs add 2^-17; FP32 sums add about 1e-6.
  Bound 1e-4.
- Prefix: weights rounded once to FP16, rms 2^-12 / sqrt(3) = 1.4e-4.  Bound
  1e-3, seven times that.
- BF16 output adds half a step, 2^-9 relative to each value.
A key within the logit error of the haze threshold may fall on either side;
its weight is e^-12 = 6e-6 of the largest, below both bounds.
"""
import math

import pytest
import torch

import kv_plain as P

pytestmark = pytest.mark.gpu
DECODE, PREFIX = 1e-4, 1e-3


@pytest.fixture(scope="module")
def dv():
    import mixed_precision_weight_b200 as pkg
    return pkg.binding


@pytest.fixture(autouse=True)
def no_device_error(dv):
    dv.dvssq_device_error(clear=True)
    yield
    assert dv.dvssq_device_error(clear=True) == 0


def to_gpu(dv, pool, table):
    return dv.KvCache(*(pool[n].cuda() for n in ("k", "v", "ks", "vs")), table.cuda())


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same_bits(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


def rows(T, H, d, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H, d), generator=g).to(torch.bfloat16)


# ------------------------------------------------------------ write and read ---
CHUNKS = [
    # (kv heads, d, start, rows per sequence)
    (4, 256, [0], [200]), (2, 128, [0, 64, 63, 1], [64, 64, 2, 130]), (2, 128, [5], [1]),
    (1, 64, [70, 0, 10], [0, 3, 61]), (8, 64, [127], [2]), (4, 256, [33, 0], [95, 0]),
    (3, 128, list(range(40)), [1 + (7 * i) % 5 for i in range(40)]),
]


@pytest.mark.parametrize("H,d,start,n", CHUNKS)
def test_append_and_read_are_exact_and_touch_nothing_else(dv, H, d, start, n):
    B, cu = len(start), [0]
    for x in n:
        cu.append(cu[-1] + x)
    T = cu[-1]
    pool, table, _ = P.filled(B, H, d, [a + b for a, b in zip(start, n)], seed=T + d)
    pool["ks"].nan_to_num_(0.5)
    pool["vs"].nan_to_num_(0.25)
    # rows are slices of a fused projection with rows behind the last sequence
    qkv = rows(T + 3, 2 + 2 * H, d, seed=T)
    k, v = qkv[:, 2:2 + H], qkv[:, 2 + H:]
    c = to_gpu(dv, pool, table)
    P.append(pool, table, k, v, start, cu)
    gq = qkv.cuda()
    dv.dvssq_kv_append(c, gq[:, 2:2 + H], gq[:, 2 + H:], i32(start), i32(cu))
    assert torch.equal(c.k.cpu(), pool["k"]) and torch.equal(c.v.cpu(), pool["v"])
    assert same_bits(c.k_scale, pool["ks"]) and same_bits(c.v_scale, pool["vs"])
    ko, vo = torch.full((T + 3, H, d), 7.0, dtype=torch.bfloat16), torch.full((T + 3, H, d), 9.0, dtype=torch.bfloat16)
    kg, vg = ko.cuda(), vo.cuda()
    P.read(pool, table, start, cu, ko, vo)
    dv.dvssq_kv_read(c, i32(start), i32(cu), T + 3, k=kg, v=vg)
    assert same_bits(kg, ko) and same_bits(vg, vo)          # the last three rows are left as they were


@pytest.mark.parametrize("H,d", [(4, 256), (2, 128), (1, 64)])
def test_single_token_form_without_cu(dv, H, d):
    start = [0, 63, 64, 100, 17]
    pool, table, _ = P.filled(5, H, d, [x + 1 for x in start], seed=d)
    pool["ks"].nan_to_num_(0.5)
    pool["vs"].nan_to_num_(0.25)
    k, v = rows(5, H, d, 1), rows(5, H, d, 2)
    c = to_gpu(dv, pool, table)
    P.append(pool, table, k, v, start, range(6))
    # head-major rows: any head and token strides
    kh = k.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    dv.dvssq_kv_append(c, kh, v.cuda(), i32(start))
    assert torch.equal(c.k.cpu(), pool["k"]) and torch.equal(c.v.cpu(), pool["v"])
    assert same_bits(c.k_scale, pool["ks"]) and same_bits(c.v_scale, pool["vs"])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    P.read(pool, table, start, range(6), ko, vo)
    kg, vg = dv.dvssq_kv_read(c, i32(start))
    assert same_bits(kg, ko) and same_bits(vg, vo)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_extreme_values(dv, d):
    """Zeros, the smallest and largest BF16 magnitudes, ties, and rows with infinities or NaN."""
    x = rows(12, 1, d, seed=d)
    x[0] = 0.0
    x[1] = 0.0
    x[1, 0, 3] = 2.0 ** -133                                # the smallest subnormal: the scale is 0
    x[2] = (x[2].float() * 2.0 ** -126).to(torch.bfloat16)  # subnormal scales
    x[3] = (x[3].float() * 2.0 ** -110).to(torch.bfloat16)
    x[4] = (x[4].float() * 2.0 ** 125).to(torch.bfloat16)
    x[5, 0, 0] = 3.3895313892515355e38                      # the largest BF16
    x[6, 0, 5] = math.inf
    x[7, 0, 1] = -math.inf
    x[8, 0, 2] = math.nan
    x[9, 0, 0], x[9, 0, 1:] = 127.0, torch.arange(1, d).to(torch.bfloat16) % 64 + 0.5   # scale 1: ties
    x[10] = -1.0
    x[11, 0, 4] = -0.0
    pool, table, _ = P.filled(1, 1, d, [12], seed=d)
    pool["ks"].nan_to_num_(0.0)
    pool["vs"].nan_to_num_(0.0)
    c = to_gpu(dv, pool, table)
    P.append(pool, table, x, x.flip(0), [0], [0, 12])
    dv.dvssq_kv_append(c, x.cuda(), x.flip(0).contiguous().cuda(), i32([0]), i32([0, 12]))
    assert torch.equal(c.k.cpu(), pool["k"]) and torch.equal(c.v.cpu(), pool["v"])
    for a, b in ((c.k_scale.cpu(), pool["ks"]), (c.v_scale.cpu(), pool["vs"])):
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
    k, _ = dv.dvssq_kv_read(c, i32([0]), i32([0, 12]), 12)
    assert k[6:9].isnan().all() and not k[:6].isnan().any() and not k[9:].isnan().any()


def test_pool_beyond_32_bit_offsets(dv):
    """Pages whose byte offsets pass 2^31 and 2^32."""
    H, d, pages = 4, 256, 70000                             # 64 KB per page and tensor
    table = i32([[69999, 40000, 3, 65536]])
    c = dv.KvCache.zeros(pages, H, d, table)
    k, v = rows(250, H, d, 5), rows(250, H, d, 6)
    dv.dvssq_kv_append(c, k.cuda(), v.cuda(), i32([0]), i32([0, 250]))
    kg, vg = dv.dvssq_kv_read(c, i32([0]), i32([0, 250]), 250)
    kc, ks = P.hold(k)
    vc, vs = P.hold(v)
    assert same_bits(kg, (kc.float() * ks.float()[..., None]).to(torch.bfloat16))
    assert same_bits(vg, (vc.float() * vs.float()[..., None]).to(torch.bfloat16))
    idx = table[0].long().cpu()
    small = dict(k=c.k[idx].cpu(), v=c.v[idx].cpu(), ks=c.k_scale[idx].cpu(), vs=c.v_scale[idx].cpu())
    q = P.queries(1, 16, d, 7)
    out = dv.dvssq_bss_attention_q8(q.cuda(), c, i32([250]))
    check(out, P.attention(q, small, torch.arange(4)[None], [250]), DECODE)


# ------------------------------------------------------------------ attention ---
def check(got, ref, bound, bf16=False):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    norm = ref.norm(dim=-1)
    err = (got - ref).norm(dim=-1)
    if bf16:
        bound = bound + 2 ** -9
    assert (err <= bound * norm).all(), float((err / norm.clamp(min=1e-300)).max())
    return float((err / norm.clamp(min=1e-300)).max())


HEADS = [(16, 4, 256), (16, 2, 128), (6, 2, 128), (8, 8, 64), (20, 4, 64), (10, 2, 256), (16, 1, 128),
         (9, 1, 64), (32, 2, 256), (7, 7, 128)]
LENS = [[1], [63, 64, 65, 0, 1], [777], [300, 2, 0, 0, 129, 128, 127]]


@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_attention_matches_plain(dv, Hq, H, d, lens):
    B = len(lens)
    q = P.queries(B, Hq, d, seed=Hq + d)
    for bind, haze in ((None, 12.0), (15.0, 12.0), (15.0, 0.0)):
        pool, table, _ = P.filled(B, H, d, lens, seed=sum(lens) + H, bind=bind and (q, bind))
        ref = P.attention(q, pool, table, lens, haze=haze)
        c = to_gpu(dv, pool, table)
        out = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), haze=haze)
        e = check(out, ref, DECODE)
        assert (out[[i for i, n in enumerate(lens) if n == 0]] == 0).all()
        print(f"Hq={Hq} H={H} d={d} lens={lens} bind={bind} haze={haze}: {e:.2e}")
        b16 = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), haze=haze, y_dtype=dv.Y_BF16)
        assert same_bits(b16, out.to(torch.bfloat16))


def test_attention_truncation_moves_the_output(dv):
    """The haze threshold is applied: with most of the context below it, the truncated result is
    matched and the untruncated one is not."""
    q = P.queries(2, 16, 128, seed=1)
    lens = [2000, 900]
    pool, table, _ = P.filled(2, 2, 128, lens, seed=2, bind=(q, 13.5))
    c = to_gpu(dv, pool, table)
    out = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens))
    ref, full = P.attention(q, pool, table, lens), P.attention(q, pool, table, lens, haze=0.0)
    e = check(out, ref, DECODE)
    first = [0, 8]                                          # the heads the keys were planted for
    miss = ((out.double().cpu() - full).norm(dim=-1) / full.norm(dim=-1))[:, first]
    assert (miss > 10 * e).all(), (miss, e)


@pytest.mark.parametrize("ctx", [3000, 9001])
def test_long_ragged_contexts(dv, ctx):
    lens = [ctx, 0, 1, ctx // 2, 64, ctx - 63]
    q = P.queries(6, 16, 128, seed=ctx)
    pool, table, _ = P.filled(6, 2, 128, lens, seed=ctx)
    out = dv.dvssq_bss_attention_q8(q.cuda(), to_gpu(dv, pool, table), i32(lens))
    check(out, P.attention(q, pool, table, lens), DECODE)


@pytest.mark.parametrize("Hq,H,d,B,ctx", [(16, 4, 256, 80, 1024), (8, 8, 64, 40, 700), (16, 1, 128, 300, 200),
                                          (6, 2, 128, 150, 960), (16, 2, 128, 2, 256), (16, 2, 128, 2, 257)])
def test_short_contexts_in_one_launch(dv, Hq, H, d, B, ctx):
    """Both sides of the rule that gives a CTA a whole sequence."""
    lens = [(131 * i + ctx) % (ctx + 1) for i in range(B)]
    lens[0], lens[1] = ctx, 0
    q = P.queries(B, Hq, d, seed=B)
    pool, table, _ = P.filled(B, H, d, lens, seed=ctx, bind=(q, 14.0))
    c = to_gpu(dv, pool, table)
    ref = P.attention(q, pool, table, lens)
    check(dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), ctx=ctx), ref, DECODE)
    # the table's capacity, one page more
    check(dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens)), ref, DECODE)


@pytest.mark.parametrize("Hq,H,d", HEADS)
def test_split_contexts_of_every_head_layout(dv, Hq, H, d):
    """Contexts past 16 pages go through the split form whatever their head layout."""
    lens = [1300, 64, 0, 1, 1025]
    q = P.queries(5, Hq, d, seed=Hq * d)
    for bind, haze in ((None, 12.0), (14.0, 12.0), (14.0, 0.0)):
        pool, table, _ = P.filled(5, H, d, lens, seed=H + 7, bind=bind and (q, bind))
        out = dv.dvssq_bss_attention_q8(q.cuda(), to_gpu(dv, pool, table), i32(lens), haze=haze)
        check(out, P.attention(q, pool, table, lens, haze=haze), DECODE)


@pytest.mark.parametrize("B", [128, 129, 300])
def test_split_form_over_many_sequences(dv, B):
    """More sequences than threads plan them, most of them short, a few of them empty or long."""
    lens = [(53 * i) % 130 for i in range(B)]
    lens[B // 2] = 1200
    q = P.queries(B, 8, 64, seed=B)
    pool, table, _ = P.filled(B, 2, 64, lens, seed=B + 1)
    c = to_gpu(dv, pool, table)
    ref = P.attention(q, pool, table, lens)
    out = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens))
    check(out, ref, DECODE)
    assert (out[[i for i, n in enumerate(lens) if n == 0]] == 0).all()


def widened(dv, pool, table, width):
    """The cache with a table of at least ``width`` pages per sequence, so that the call's bound on the
    lengths, which picks the kernels, is that of a long context."""
    more = torch.full((table.shape[0], max(0, width - table.shape[1])), -9, dtype=torch.int32)
    return to_gpu(dv, pool, torch.cat([table, more], 1).contiguous())


@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("lens", [[1300, 64, 0, 1, 1025], [513, 0, 512], [2100], [3000, 3, 4096], [70] * 33 + [0, 900]],
                         ids=lambda x: f"B{len(x)}_{max(x)}")
def test_every_form_of_every_head_layout(dv, Hq, H, d, lens):
    """The same sequences with bounds of 1 x, 17, 33, 65 and 129 pages: one CTA, clusters, three launches."""
    B = len(lens)
    q = P.queries(B, Hq, d, seed=Hq + d)
    for bind, haze in ((None, 12.0), (14.0, 0.0)):
        pool, table, _ = P.filled(B, H, d, lens, seed=H + B, bind=bind and (q, bind))
        ref = P.attention(q, pool, table, lens, haze=haze)
        for width in (0, 17, 33, 65, 129):
            c = widened(dv, pool, table, width)
            out = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), haze=haze)
            check(out, ref, DECODE)
            assert torch.equal(out, dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), haze=haze))
            b16 = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), haze=haze, y_dtype=dv.Y_BF16)
            assert same_bits(b16, out.to(torch.bfloat16))


@pytest.mark.parametrize("B", [128, 129, 300])
@pytest.mark.parametrize("width", [20, 65])
def test_long_bounds_over_many_sequences(dv, B, width):
    """As test_split_form_over_many_sequences under a table of more pages than any sequence has."""
    lens = [(53 * i) % 130 for i in range(B)]
    lens[B // 2] = 1200
    q = P.queries(B, 8, 128, seed=B)
    pool, table, _ = P.filled(B, 2, 128, lens, seed=B + 2)
    out = dv.dvssq_bss_attention_q8(q.cuda(), widened(dv, pool, table, width), i32(lens))
    check(out, P.attention(q, pool, table, lens), DECODE)
    assert (out[[i for i, n in enumerate(lens) if n == 0]] == 0).all()


def test_nan_rows_in_every_form(dv):
    """A sequence of NaN rows is NaN and its neighbours are not, whatever kernels run."""
    lens = [700, 100, 0]
    q = P.queries(3, 8, 128, seed=41)
    pool, table, _ = P.filled(3, 2, 128, lens, seed=42)
    ref = P.attention(q, pool, table, lens)
    for p in table[0, :11].tolist():
        pool["ks"][p] = math.nan
    for width in (0, 17, 40, 65):
        out = dv.dvssq_bss_attention_q8(q.cuda(), widened(dv, pool, table, width), i32(lens)).cpu()
        assert out[0].isnan().all()
        check(out[1:], ref[1:], DECODE)


def test_many_short_sequences(dv):
    lens = [(37 * i) % 90 for i in range(600)]
    q = P.queries(600, 4, 64, seed=3)
    pool, table, _ = P.filled(600, 2, 64, lens, seed=4)
    c = to_gpu(dv, pool, table)
    check(dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens)), P.attention(q, pool, table, lens), DECODE)


def test_query_strides_context_bound_and_determinism(dv):
    lens = [500, 90, 301]
    q = P.queries(3, 16, 128, seed=9)
    pool, table, _ = P.filled(3, 4, 128, lens, seed=10)
    c = to_gpu(dv, pool, table)
    ref = P.attention(q, pool, table, lens)
    a = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens))
    check(a, ref, DECODE)
    fused = torch.randn((3, 24, 128), device="cuda").to(torch.bfloat16)
    fused[:, :16] = q.cuda()
    b = dv.dvssq_bss_attention_q8(fused[:, :16], c, i32(lens))
    assert torch.equal(a, b)
    hm = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    assert torch.equal(a, dv.dvssq_bss_attention_q8(hm, c, i32(lens)))
    # a tighter bound on the lengths gives the same keys to the same sums
    t = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), ctx=500)
    check(t, ref, DECODE)
    ws = torch.empty(dv.dvssq_bss_attention_q8_workspace_size(dv.AttnShape(3, 16, 4, 128, 576, 1.1, 12.0)),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(255)                                            # the workspace's old contents do not matter
    out = torch.empty((3, 16, 128), device="cuda")
    assert torch.equal(a, dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), ctx=576, out=out, workspace=ws))
    assert torch.equal(a, dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens), ctx=576, out=out, workspace=ws))


def test_extreme_queries_and_keys(dv):
    """A zero query, queries of tiny and large magnitude, keys that read back as zero."""
    lens = [130]
    q = P.queries(1, 4, 128, seed=11)
    q[0, 0] = 0.0
    q[0, 1] = (q[0, 1].float() * 2.0 ** -120).to(torch.bfloat16)
    q[0, 2, 5:] = 0.0
    q[0, 2, :5] = torch.tensor([255.0, -255.0, 1.9921875, 0.0078125, -3.0]).to(torch.bfloat16)
    pool, table, _ = P.filled(1, 1, 128, lens, seed=12, std=0.25)
    page = int(table[0, 0])
    pool["ks"][page, 0, 3] = 0.0
    pool["vs"][page, 0, 4] = 0.0
    c = to_gpu(dv, pool, table)
    out = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens))
    check(out, P.attention(q, pool, table, lens), 5e-4)     # max|q| = 255 beside small values: logits near 60


@pytest.mark.parametrize("prefix", [0, 1, 64])
def test_a_context_of_nan_rows_is_nan(dv, prefix):
    """Where every key of a sequence reads back as NaN, so does its output."""
    lens = [1, 3, 0]
    q = P.queries(3, 4, 64, seed=16)
    pool, table, ptable = P.filled(3, 2, 64, lens, seed=17, prefix=prefix)
    pool["ks"][:] = math.nan
    c = to_gpu(dv, pool, table)
    if prefix:
        out = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), ptable.cuda(), prefix)
        assert out.isnan().all()
    else:
        out = dv.dvssq_bss_attention_q8(q.cuda(), c, i32(lens))
        assert out[:2].isnan().all() and (out[2] == 0).all()


def test_nan_rows_reach_only_their_own_head(dv):
    """A NaN key row makes its KV head's outputs NaN; a NaN value row does so only where its
    weight is kept; a NaN query head stays in its head."""
    lens = [200, 100]
    q = P.queries(2, 8, 128, seed=13)
    pool, table, _ = P.filled(2, 4, 128, lens, seed=14)
    ref = P.attention(q, pool, table, lens)
    pool["ks"][int(table[0, 1]), 2, 7] = math.nan
    pool["vs"][int(table[1, 0]), 1, 9] = math.nan
    qn = q.clone()
    qn[1, 7, 3] = math.nan
    out = dv.dvssq_bss_attention_q8(qn.cuda(), to_gpu(dv, pool, table), i32(lens)).cpu()
    bad = torch.zeros((2, 8), dtype=torch.bool)
    bad[0, 4:6] = True
    bad[1, 2:4] = True
    bad[1, 7] = True
    assert out[bad].isnan().all()
    good = ~bad
    assert (out[good].double() - ref[good]).norm() <= DECODE * ref[good].norm()


# --------------------------------------------------------------------- prefix ---
PREFIXES = [(16, 4, 256, [5, 0, 64], 129), (16, 2, 128, [0], 64), (6, 2, 128, [3, 70, 1, 0, 65], 300),
            (8, 8, 64, [17] * 20, 1), (20, 4, 64, [1, 2], 63), (10, 2, 256, [100, 0], 200),
            (16, 1, 128, [9] * 9, 513), (16, 4, 256, [0] * 33, 777), (32, 2, 256, [30, 0, 2], 65),
            (16, 2, 128, [10, 80], 0), (7, 7, 128, [0, 1], 128), (9, 1, 64, [4] * 40, 1500)]


@pytest.mark.parametrize("Hq,H,d,lens,prefix", PREFIXES)
def test_prefix_matches_plain(dv, Hq, H, d, lens, prefix):
    B = len(lens)
    q = P.queries(B, Hq, d, seed=prefix + d)
    for bind, haze in ((None, 12.0), (15.0, 12.0), (15.0, 0.0)):
        pool, table, ptable = P.filled(B, H, d, lens, seed=prefix, prefix=prefix, bind=bind and (q, bind))
        ref = P.attention(q, pool, table, lens, haze=haze, ptable=ptable, prefix=prefix)
        c = to_gpu(dv, pool, table)
        args = (q.cuda(), c, i32(lens), ptable.cuda(), prefix)
        out = dv.dvssq_bss_attention_prefix(*args, haze=haze)
        e = check(out, ref, PREFIX)
        print(f"Hq={Hq} H={H} d={d} B={B} prefix={prefix} bind={bind} haze={haze}: {e:.2e}")
        b16 = dv.dvssq_bss_attention_prefix(*args, haze=haze, y_dtype=dv.Y_BF16)
        assert same_bits(b16, out.to(torch.bfloat16))
        assert torch.equal(out, dv.dvssq_bss_attention_prefix(*args, haze=haze))


def test_prefix_longer_with_uneven_value_scales(dv):
    """Value rows whose scales span four orders of magnitude, on a prefix of many tiles."""
    lens, prefix = [33, 0, 200], 4100
    q = P.queries(3, 16, 128, seed=20)
    pool, table, ptable = P.filled(3, 2, 128, lens, seed=21, prefix=prefix)
    g = torch.Generator().manual_seed(22)
    f = torch.exp(torch.empty(pool["vs"].shape).uniform_(-9.0, 0.0, generator=g))
    pool["vs"] = (pool["vs"].float() * f).to(torch.bfloat16)
    c = to_gpu(dv, pool, table)
    out = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), ptable.cuda(), prefix)
    check(out, P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix), PREFIX)


def test_prefix_with_tiny_value_scales(dv):
    """Value scales near 2^-110: the power of two that lifts the weights ends at 2^100, so that
    their sum stays finite.  The largest weight is then about 2^-11, in FP16 steps of at
    least 2^-24: sqrt(300) 2^-25 / sqrt(3) over 2^-11 is 6e-4, beside the rounding's 1.4e-4;
    bound 2e-3."""
    lens, prefix = [3, 0], 300
    q = P.queries(2, 16, 128, seed=25)
    pool, table, ptable = P.filled(2, 4, 128, lens, seed=26, prefix=prefix)
    pool["vs"] = (pool["vs"].float() * 2.0 ** -105).to(torch.bfloat16)
    c = to_gpu(dv, pool, table)
    out = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), ptable.cuda(), prefix).cpu()
    ref = P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix)
    check(out.double() * 2.0 ** 105, ref * 2.0 ** 105, 2e-3)


def test_scalars_as_tensors_and_the_default_stream(dv):
    """tau held in a tensor that changes between calls is read anew; stream 0 is the default stream."""
    lens = [70]
    q = P.queries(1, 8, 64, seed=27).cuda()
    pool, table, _ = P.filled(1, 2, 64, lens, seed=28)
    c, lg, tau = to_gpu(dv, pool, table), i32(lens), torch.tensor(1.0)
    a = dv.dvssq_bss_attention_q8(q, c, lg, tau=tau)
    assert torch.equal(a, dv.dvssq_bss_attention_q8(q, c, lg, tau=1.0))
    tau.fill_(2.0)
    b = dv.dvssq_bss_attention_q8(q, c, lg, tau=tau, stream=torch.cuda.default_stream())
    assert torch.equal(b, dv.dvssq_bss_attention_q8(q, c, lg, tau=2.0, stream=0)) and not torch.equal(a, b)


# Enough visits (sequences x KV heads x pages) that the prefix is read once for all sequences.
SHARED = [(16, 4, 256, [5, 0, 64] * 6, 4100), (16, 2, 128, [0, 70, 1] * 12, 3800),
          (6, 2, 128, [3, 70, 1, 0, 65] * 10, 2625), (8, 8, 64, [17] * 40, 897), (20, 4, 64, [1, 2] * 40, 1000),
          (10, 2, 256, [100, 0] * 20, 3500), (16, 1, 128, [9] * 60, 2700), (32, 2, 256, [30, 0, 2] * 10, 2600),
          (7, 7, 128, [0, 1] * 300, 64), (7, 7, 64, [0, 3] * 300, 1), (14, 7, 64, [1, 0] * 300, 63),
          (5, 5, 128, [1, 0] * 250, 129), (9, 1, 64, [4, 0] * 650, 100), (16, 4, 128, [1500, 0, 7] * 6, 3800)]


@pytest.mark.parametrize("Hq,H,d,lens,prefix", SHARED)
def test_prefix_read_once_matches_plain(dv, Hq, H, d, lens, prefix):
    B = len(lens)
    assert B * H * -(-prefix // 64) > (4096 if Hq // H <= 8 else 2400)
    q = P.queries(B, Hq, d, seed=prefix + d)
    for bind, haze in ((None, 12.0), (15.0, 12.0), (15.0, 0.0)):
        pool, table, ptable = P.filled(B, H, d, lens, seed=prefix, prefix=prefix, bind=bind and (q, bind))
        ref = P.attention(q, pool, table, lens, haze=haze, ptable=ptable, prefix=prefix)
        c = to_gpu(dv, pool, table)
        args = (q.cuda(), c, i32(lens), ptable.cuda(), prefix)
        out = dv.dvssq_bss_attention_prefix(*args, haze=haze)
        check(out, ref, PREFIX)
        b16 = dv.dvssq_bss_attention_prefix(*args, haze=haze, y_dtype=dv.Y_BF16)
        assert same_bits(b16, out.to(torch.bfloat16))
        assert torch.equal(out, dv.dvssq_bss_attention_prefix(*args, haze=haze))


def test_prefix_read_once_with_uneven_and_tiny_value_scales(dv):
    """As the two tests above; tiny scales: sqrt(1000) 2^-25 / sqrt(3) over 2^-11 is 1.1e-3, bound 3e-3."""
    lens, prefix = [33, 0, 200] * 12, 4100
    q = P.queries(36, 16, 128, seed=20)
    pool, table, ptable = P.filled(36, 2, 128, lens, seed=21, prefix=prefix)
    g = torch.Generator().manual_seed(22)
    f = torch.exp(torch.empty(pool["vs"].shape).uniform_(-9.0, 0.0, generator=g))
    pool["vs"] = (pool["vs"].float() * f).to(torch.bfloat16)
    out = dv.dvssq_bss_attention_prefix(q.cuda(), to_gpu(dv, pool, table), i32(lens), ptable.cuda(), prefix)
    check(out, P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix), PREFIX)
    lens, prefix = [3, 0] * 40, 1000
    q = P.queries(80, 16, 128, seed=25)
    pool, table, ptable = P.filled(80, 4, 128, lens, seed=26, prefix=prefix)
    pool["vs"] = (pool["vs"].float() * 2.0 ** -105).to(torch.bfloat16)
    out = dv.dvssq_bss_attention_prefix(q.cuda(), to_gpu(dv, pool, table), i32(lens), ptable.cuda(), prefix).cpu()
    check(out.double() * 2.0 ** 105, P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix) * 2.0 ** 105, 3e-3)


def test_prefix_read_once_nan_rows_and_bad_pages(dv):
    lens, prefix = [1, 3, 0] * 100, 1000
    q = P.queries(300, 4, 64, seed=16)
    pool, table, ptable = P.filled(300, 2, 64, lens, seed=17, prefix=prefix)
    pool["ks"].nan_to_num_(0.01)
    pool["vs"].nan_to_num_(0.01)
    c = to_gpu(dv, pool, table)
    bad = ptable.clone()
    bad[15] = pool["k"].shape[0]                             # the last 40 keys
    out = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), bad.cuda(), prefix)
    assert dv.dvssq_device_error(clear=True) == 16
    check(out, P.attention(q, pool, table, lens, ptable=ptable, prefix=960), PREFIX)
    pool["ks"][int(ptable[3]), 1, 5] = math.nan
    out = dv.dvssq_bss_attention_prefix(q.cuda(), to_gpu(dv, pool, table), i32(lens), ptable.cuda(), prefix).cpu()
    assert out[:, 2:].isnan().all()
    pool["ks"][int(ptable[3]), 1, 5] = 0.01
    check(out[:, :2], P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix)[:, :2], PREFIX)
    pool["ks"][:] = math.nan
    assert dv.dvssq_bss_attention_prefix(q.cuda(), to_gpu(dv, pool, table), i32(lens), ptable.cuda(), prefix).isnan().all()


@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("prefix,lens", [(1000, [70, 0, 300]), (4000, [0, 130, 5]), (6000, [2000]), (65, [1, 0])])
def test_prefix_as_first_keys(dv, Hq, H, d, prefix, lens):
    """Prefixes of few visits, in one launch and in three: the arithmetic of the form without a prefix."""
    B = len(lens)
    q = P.queries(B, Hq, d, seed=prefix)
    for bind in (None, 14.0):
        pool, table, ptable = P.filled(B, H, d, lens, seed=prefix + H, prefix=prefix, bind=bind and (q, bind))
        out = dv.dvssq_bss_attention_prefix(q.cuda(), to_gpu(dv, pool, table), i32(lens), ptable.cuda(), prefix)
        check(out, P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix), DECODE)


@pytest.mark.parametrize("lens,prefix", [([1500, 0, 7], 300), ([5000], 64), ([0, 0], 700), ([1025] * 9, 129)])
def test_prefix_before_long_own_contexts(dv, lens, prefix):
    """Own contexts that are split over CTAs (and tables that allow it without using it)."""
    B = len(lens)
    q = P.queries(B, 16, 128, seed=sum(lens) + B)
    for bind in (None, 13.0):
        pool, table, ptable = P.filled(B, 4, 128, lens, seed=prefix, prefix=prefix, bind=bind and (q, bind))
        wide = torch.cat([table, torch.full((B, 17), -7, dtype=torch.int32)], 1)
        c = to_gpu(dv, pool, wide)
        out = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), ptable.cuda(), prefix)
        check(out, P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix), PREFIX)
        again = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), ptable.cuda(), prefix)
        assert torch.equal(out, again)


def test_prefix_equals_the_same_keys_in_the_own_table(dv):
    """A page-aligned prefix gives what the decode form gives over the joined page lists."""
    lens, prefix = [40, 7], 256
    q = P.queries(2, 16, 128, seed=23)
    pool, table, ptable = P.filled(2, 4, 128, lens, seed=24, prefix=prefix)
    c = to_gpu(dv, pool, table)
    a = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32(lens), ptable.cuda(), prefix)
    joined = torch.cat([ptable[None].expand(2, -1), table], 1).contiguous()
    cj = dv.KvCache(c.k, c.v, c.k_scale, c.v_scale, joined.cuda())
    b = dv.dvssq_bss_attention_q8(q.cuda(), cj, i32([n + prefix for n in lens]))
    assert ((a - b).norm(dim=-1) <= (PREFIX + DECODE) * b.norm(dim=-1)).all()


# ------------------------------------------------------------------- together ---
def test_decode_loop_in_a_graph(dv):
    """A prompt is written, then ten captured steps append one token per sequence and attend:
    every step equals the plain implementation on the growing cache."""
    B, Hq, H, d = 3, 16, 4, 128
    prompt = [60, 5, 127]
    steps = 10
    pool, table, _ = P.filled(B, H, d, [n + steps for n in prompt], seed=30)
    for n in ("ks", "vs"):
        pool[n].zero_()
    c = to_gpu(dv, pool, table)
    cu = [0, 60, 65, 192]
    k, v = rows(192, H, d, 31), rows(192, H, d, 32)
    P.append(pool, table, k, v, [0] * B, cu)
    dv.dvssq_kv_append(c, k.cuda(), v.cuda(), i32([0] * B), i32(cu))
    qkv = torch.zeros((B, Hq + 2 * H, d), dtype=torch.bfloat16, device="cuda")
    pos, lens = i32(prompt), i32([n + 1 for n in prompt])

    def step():
        dv.dvssq_kv_append(c, qkv[:, Hq:Hq + H], qkv[:, Hq + H:], pos)
        return dv.dvssq_bss_attention_q8(qkv[:, :Hq], c, lens)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()                                              # the first token, eagerly on a side stream
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(steps):
        new = rows(B, Hq + 2 * H, d, 40 + i)
        qkv.copy_(new.cuda())
        graph.replay()
        at = [n + i for n in prompt]
        P.append(pool, table, new[:, Hq:Hq + H], new[:, Hq + H:], at, range(B + 1))
        check(out, P.attention(new[:, :Hq], pool, table, [n + 1 for n in at]), DECODE)
        pos.add_(1)
        lens.add_(1)
    torch.cuda.synchronize()
    assert torch.equal(c.k.cpu(), pool["k"]) and torch.equal(c.v.cpu(), pool["v"])
    assert same_bits(c.k_scale, pool["ks"]) and same_bits(c.v_scale, pool["vs"])


def test_shared_prefix_loop(dv):
    """The prefix is written once through its own cache object over the same pool; samples then
    grow behind it; the keys read back attend to the same result."""
    B, Hq, H, d, prefix, steps = 5, 16, 2, 128, 150, 4
    pool, table, ptable = P.filled(B, H, d, [steps] * B, seed=50, prefix=prefix)
    for n in ("ks", "vs"):
        pool[n].zero_()
    c = to_gpu(dv, pool, table)
    doc = dv.KvCache(c.k, c.v, c.k_scale, c.v_scale, ptable[None].contiguous().cuda())
    k, v = rows(prefix, H, d, 51), rows(prefix, H, d, 52)
    P.append(pool, ptable[None], k, v, [0], [0, prefix])
    dv.dvssq_kv_append(doc, k.cuda(), v.cuda(), i32([0]), i32([0, prefix]))
    for i in range(steps):
        q, kn, vn = P.queries(B, Hq, d, 60 + i), rows(B, H, d, 70 + i), rows(B, H, d, 80 + i)
        P.append(pool, table, kn, vn, [i] * B, range(B + 1))
        dv.dvssq_kv_append(c, kn.cuda(), vn.cuda(), i32([i] * B))
        out = dv.dvssq_bss_attention_prefix(q.cuda(), c, i32([i + 1] * B), ptable.cuda(), prefix)
        check(out, P.attention(q, pool, table, [i + 1] * B, ptable=ptable, prefix=prefix), PREFIX)
    ko, vo = dv.dvssq_kv_read(doc, i32([0]), i32([0, prefix]), prefix)
    kp, vp = P.keys_values(pool, ptable, prefix)
    assert same_bits(ko, kp.transpose(0, 1).float().to(torch.bfloat16).contiguous())
    assert same_bits(vo, vp.transpose(0, 1).float().to(torch.bfloat16).contiguous())


def test_index_arrays_may_be_slices(dv):
    """Index arrays at any 4-byte offset, as slices of one tensor give them."""
    lens, prefix = [70, 0, 5], 100
    q = P.queries(3, 8, 64, seed=85)
    pool, table, ptable = P.filled(3, 2, 64, lens, seed=86, prefix=prefix)
    flat = torch.cat([i32([0]), table.reshape(-1).cuda(), i32([0]), ptable.cuda(), i32([0] + lens)])
    at, W = 1, table.shape[1]
    views = []
    for n in (3 * W, 2, 3):
        views.append(flat[at: at + n])
        at += n + 1
    assert all(x.data_ptr() % 16 for x in views[:2])
    c = dv.KvCache(*(pool[n].cuda() for n in ("k", "v", "ks", "vs")), views[0].view(3, W))
    out = dv.dvssq_bss_attention_prefix(q.cuda(), c, views[2], views[1], prefix)
    check(out, P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix), PREFIX)


def test_two_streams_and_explicit_streams(dv):
    """Calls on two streams at once, each with its own workspace, give what one stream gives."""
    lens = [1200, 700]
    q = P.queries(2, 16, 128, seed=90)
    pool, table, _ = P.filled(2, 2, 128, lens, seed=91)
    c, lg, qg = to_gpu(dv, pool, table), i32(lens), q.cuda()
    ref = dv.dvssq_bss_attention_q8(qg, c, lg)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [dv.dvssq_bss_attention_q8(qg, c, lg, stream=s) for _ in range(5)
            for s in (s1, s2, s1.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_two_graphs_share_a_workspace_one_after_the_other(dv):
    lens_a, lens_b = [300, 0], [64, 500]
    q = P.queries(2, 8, 128, seed=92)
    pool, table, _ = P.filled(2, 4, 128, [300, 500], seed=93)
    c, qg = to_gpu(dv, pool, table), q.cuda()
    shape = dv.AttnShape(2, 8, 4, 128, 64 * table.shape[1], 1.1, 12.0)
    ws = torch.empty(dv.dvssq_bss_attention_q8_workspace_size(shape), dtype=torch.uint8, device="cuda")
    la, lb = i32(lens_a), i32(lens_b)
    want = [dv.dvssq_bss_attention_q8(qg, c, x).clone() for x in (la, lb)]
    graphs, outs = [], []
    for x in (la, lb):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dv.dvssq_bss_attention_q8(qg, c, x, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


# ------------------------------------------------------------------- refusals ---
def test_binding_refusals(dv):
    pool, table, ptable = P.filled(2, 2, 128, [100, 30], seed=95, prefix=70)
    c = to_gpu(dv, pool, table)
    q, lens = P.queries(2, 4, 128, 1).cuda(), i32([100, 30])
    k = rows(2, 2, 128, 2).cuda()
    with pytest.raises(ValueError):
        dv.dvssq_kv_append(c, k, k.cpu(), i32([0, 0]))
    with pytest.raises(TypeError):
        dv.dvssq_kv_append(c, k.float(), k, i32([0, 0]))
    with pytest.raises(TypeError):
        dv.dvssq_kv_append(c, k, k, torch.tensor([0, 0], device="cuda"))
    with pytest.raises(ValueError):
        dv.dvssq_kv_append(c, k, k, i32([0, 0, 0]))
    with pytest.raises(ValueError):
        dv.dvssq_kv_append(c, k, k, i32([0, 0]), i32([0, 2]))
    with pytest.raises(dv.DvssqError):                       # three rows, two sequences, no cu
        dv.dvssq_kv_append(c, rows(3, 2, 128, 2).cuda(), rows(3, 2, 128, 2).cuda(), i32([0, 0]))
    with pytest.raises(ValueError):
        dv.dvssq_kv_read(c, i32([0, 0]), i32([0, 1, 2]))
    with pytest.raises(ValueError):
        dv.dvssq_kv_read(c, i32([0, 0]), k=torch.empty((2, 2, 128), device="cuda"))
    with pytest.raises(ValueError):
        dv.dvssq_bss_attention_q8(q[:1], c, lens)
    with pytest.raises(ValueError):
        dv.dvssq_bss_attention_q8(q, c, lens.cpu())
    with pytest.raises(ValueError):
        dv.dvssq_bss_attention_q8(q, c, lens, out=torch.empty((2, 4, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        dv.dvssq_bss_attention_q8(q, c, lens, y_dtype=5)
    with pytest.raises(dv.DvssqError):
        dv.dvssq_bss_attention_q8(q, c, lens, ctx=10 ** 6)   # longer than the table
    with pytest.raises(dv.DvssqError):
        dv.dvssq_bss_attention_prefix(q, widened(dv, pool, table, 65), lens, ptable.cuda(), 70,
                                      workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        dv.dvssq_bss_attention_prefix(q, c, lens, ptable.cuda(), 200)
    with pytest.raises(ValueError):
        dv.dvssq_bss_attention_prefix(q, c, lens, ptable[:0].cuda(), -1)


def test_bad_indices_are_flagged_and_skipped(dv):
    """Indices out of range, which only the kernels can see: bit 4 of the error word, the rest right."""
    pool, table, ptable = P.filled(2, 2, 128, [100, 130], seed=96, prefix=130)
    pool["ks"].nan_to_num_(0.5)
    pool["vs"].nan_to_num_(0.25)
    q = P.queries(2, 4, 128, 97)
    ref = P.attention(q, pool, table, [100, 130])
    good = to_gpu(dv, pool, table)

    def flagged():
        return dv.dvssq_device_error(clear=True) == 16

    # a page outside the pool: its keys are left out (the last 36 of sequence 0)
    bad = table.clone()
    bad[0, 1] = pool["k"].shape[0]
    cb = dv.KvCache(good.k, good.v, good.k_scale, good.v_scale, bad.cuda())
    out = dv.dvssq_bss_attention_q8(q.cuda(), cb, i32([100, 130]))
    assert flagged()
    want = P.attention(q, pool, table, [64, 130])
    check(out, want, DECODE)
    # a negative page in the shared prefix
    pb = ptable.clone()
    pb[2] = -1
    out = dv.dvssq_bss_attention_prefix(q.cuda(), good, i32([100, 130]), pb.cuda(), 130)
    assert flagged()
    check(out, P.attention(q, pool, table, [100, 130], ptable=ptable, prefix=128), PREFIX)
    # lengths outside [0, ctx] are clamped
    out = dv.dvssq_bss_attention_q8(q.cuda(), good, i32([-5, 130]), ctx=130)
    assert flagged() and (out[0] == 0).all()
    check(out[1:], ref[1:], DECODE)
    out = dv.dvssq_bss_attention_q8(q.cuda(), good, i32([100, 2 ** 31 - 1]), ctx=130)
    assert flagged()
    check(out, ref, DECODE)
    # rows at negative positions, past the table, in pages outside the pool, past the call's rows
    k = rows(4, 2, 128, 98).cuda()
    width = 64 * table.shape[1]
    for c, start, cu in ((good, [-1, 0], [0, 1, 1]), (good, [width, 0], [0, 4, 4]), (cb, [64, 0], [0, 4, 4])):
        before = c.k.clone()
        dv.dvssq_kv_append(c, k, k, i32(start), i32(cu))
        assert flagged() and torch.equal(c.k, before)
        mark = torch.full((4, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        dv.dvssq_kv_read(c, i32(start), i32(cu), 4, k=mark, v=mark.clone())
        assert flagged() and (mark == 3.0).all()
    dv.dvssq_kv_append(good, k, k, i32([0, 0]), i32([0, 0, 9]))
    assert flagged()
    P.append(pool, table, k.cpu(), k.cpu(), [0, 0], [0, 0, 4])
    assert torch.equal(good.k.cpu(), pool["k"]) and torch.equal(good.v.cpu(), pool["v"])
