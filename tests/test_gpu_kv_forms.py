"""The forms of KV-BSS attention over the 8-bit cache that keep logits, maxima, partial sums and
offsets in a workspace: three launches over long contexts, and a prefix read once with short
and with long own contexts behind it (five launches).  Tables are wide enough, and prefixes
long enough, that these forms run; every test asserts it.  Against the plain 64-bit
implementation (kv_plain.py), with the bounds of test_gpu_kv_cache.py.
"""
import pytest
import torch

import kv_plain as P
from test_gpu_kv_cache import DECODE, HEADS, PREFIX, check, i32, to_gpu, widened

pytestmark = pytest.mark.gpu
WIDE = 130                       # pages of the table: beyond every one-launch form


@pytest.fixture(scope="module")
def dv():
    import mixed_precision_weight_b200 as pkg
    return pkg.binding


@pytest.fixture(autouse=True)
def no_device_error(dv):
    dv.dvssq_device_error(clear=True)
    yield
    assert dv.dvssq_device_error(clear=True) == 0


def once(B, H, G, prefix):
    """Whether the prefix is read once (the header's rule)."""
    return B * H * -(-prefix // 64) > (4096 if G <= 8 else 2400)


class Decode:
    """A call over long contexts: table wide enough for three launches."""

    def __init__(self, dv, Hq, H, d, lens, seed, width=WIDE, bind=None, haze=12.0):
        B = len(lens)
        self.dv, self.lens, self.haze = dv, lens, haze
        self.q = P.queries(B, Hq, d, seed=seed)
        self.pool, self.table, _ = P.filled(B, H, d, lens, seed=seed + 1, bind=bind and (self.q, bind))
        self.cache = widened(dv, self.pool, self.table, width)
        self.args = (self.q.cuda(), self.cache, i32(lens))
        self.need = dv.dvssq_bss_attention_q8_workspace_size(
            dv.AttnShape(B, Hq, H, d, 64 * self.cache.width, 1.1, haze))
        assert self.need > 0
        self.bound = DECODE

    def __call__(self, **kw):
        return self.dv.dvssq_bss_attention_q8(*self.args, haze=self.haze, **kw)

    def ref(self):
        return P.attention(self.q, self.pool, self.table, self.lens, haze=self.haze)


class Prefix(Decode):
    """A call whose prefix is read once; ``split``: the bound on the own lengths is beyond 16 pages."""

    def __init__(self, dv, Hq, H, d, lens, prefix, seed, split, bind=None, haze=12.0):
        B = len(lens)
        assert once(B, H, Hq // H, prefix)
        self.dv, self.lens, self.haze, self.prefix = dv, lens, haze, prefix
        self.q = P.queries(B, Hq, d, seed=seed)
        self.pool, self.table, self.ptable = P.filled(B, H, d, lens, seed=seed + 1, prefix=prefix,
                                                      bind=bind and (self.q, bind))
        self.cache = widened(dv, self.pool, self.table, 17 if split else 0)
        assert (self.cache.width > 16) == split
        self.args = (self.q.cuda(), self.cache, i32(lens), self.ptable.cuda(), prefix)
        self.need = dv.dvssq_bss_attention_prefix_workspace_size(
            dv.AttnShape(B, Hq, H, d, 64 * self.cache.width, 1.1, haze), prefix)
        assert self.need > 0
        self.bound = PREFIX

    def __call__(self, **kw):
        return self.dv.dvssq_bss_attention_prefix(*self.args, haze=self.haze, **kw)

    def ref(self):
        return P.attention(self.q, self.pool, self.table, self.lens, haze=self.haze, ptable=self.ptable,
                           prefix=self.prefix)


KINDS = {
    "decode": lambda dv, seed: Decode(dv, 16, 2, 128, [2100, 0, 700, 64], seed),
    "prefix_short": lambda dv, seed: Prefix(dv, 16, 4, 128, [40, 0, 65] * 6, 3800, seed, False),
    "prefix_split": lambda dv, seed: Prefix(dv, 16, 4, 128, [1200, 0, 7] * 6, 3800, seed, True),
}


# ---------------------------------------------------------------- head layouts ---
@pytest.mark.parametrize("Hq,H,d", HEADS)
def test_three_launches_of_every_head_layout(dv, Hq, H, d):
    for bind, haze in ((None, 12.0), (14.0, 12.0), (14.0, 0.0)):
        c = Decode(dv, Hq, H, d, [1300, 64, 0, 1, 1025, 3000], seed=Hq * d, bind=bind, haze=haze)
        out = c()
        check(out, c.ref(), DECODE)
        assert (out[2] == 0).all() and torch.equal(out, c())
        assert torch.equal(c(y_dtype=dv.Y_BF16), out.to(torch.bfloat16))


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("B", [1, 127, 128, 129, 300])
def test_three_launches_over_many_sequences(dv, B, d):
    """More sequences than the threads that plan them; most of them short, some empty, one long."""
    lens = [(53 * i) % 130 for i in range(B)]
    lens[B // 2] = 1200
    c = Decode(dv, 8, 2, d, lens, seed=B)
    out = c()
    check(out, c.ref(), DECODE)
    assert (out[[i for i, n in enumerate(lens) if n == 0]] == 0).all()


@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("split", [False, True])
def test_prefix_read_once_of_every_head_layout(dv, Hq, H, d, split):
    """Short own contexts (beside the maximum pass) and long ones (items), with empty sequences."""
    lens = [1100, 0, 7, 64, 1025, 130, 1] if split else [100, 0, 7, 64, 0, 130, 1]
    prefix = 64 * ((4096 if Hq // H <= 8 else 2400) // (7 * H) + 1) - 27
    for bind, haze in ((None, 12.0), (14.0, 0.0)):
        c = Prefix(dv, Hq, H, d, lens, prefix, Hq + d, split, bind=bind, haze=haze)
        out = c()
        check(out, c.ref(), PREFIX)
        assert torch.equal(out, c())
        assert torch.equal(c(y_dtype=dv.Y_BF16), out.to(torch.bfloat16))


@pytest.mark.parametrize("split", [False, True])
def test_prefix_read_once_without_own_keys(dv, split):
    c = Prefix(dv, 16, 4, 256, [0] * 12, 5600, 3, split)
    check(c(), c.ref(), PREFIX)


# ------------------------------------------------------------------ workspaces ---
@pytest.mark.parametrize("kind", KINDS)
def test_old_contents_of_the_workspace_do_not_matter(dv, kind):
    c = KINDS[kind](dv, 11)
    want = c()
    check(want, c.ref(), c.bound)
    ws = torch.full((c.need,), 255, dtype=torch.uint8, device="cuda")       # NaN in every float
    assert torch.equal(want, c(workspace=ws)) and torch.equal(want, c(workspace=ws))
    with pytest.raises(dv.DvssqError):
        c(workspace=ws[: c.need - 256])


@pytest.mark.parametrize("a", KINDS)
@pytest.mark.parametrize("b", KINDS)
def test_one_workspace_for_calls_of_two_shapes(dv, a, b):
    """The larger call, then the smaller, then the larger again over the same bytes, in a row."""
    x, y = KINDS[a](dv, 21), KINDS[b](dv, 22)
    wx, wy = x(), y()
    ws = torch.full((max(x.need, y.need),), 255, dtype=torch.uint8, device="cuda")
    got = [f(workspace=ws) for _ in range(3) for f in (x, y)]
    assert all(torch.equal(g, w) for g, w in zip(got, [wx, wy] * 3))


@pytest.mark.parametrize("a", KINDS)
@pytest.mark.parametrize("b", KINDS)
def test_two_graphs_share_a_workspace(dv, a, b):
    """Replayed one after the other and with eager calls between them."""
    x, y = KINDS[a](dv, 31), KINDS[b](dv, 32)
    want = [x().clone(), y().clone()]
    ws = torch.full((max(x.need, y.need),), 255, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c(workspace=ws))
        graphs.append(g)
    for i in range(4):
        for g in graphs:
            g.replay()
            if i & 1:
                x(workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("kind", KINDS)
def test_streams_with_their_own_workspaces(dv, kind):
    """Calls in flight on three streams at once give what one stream gives."""
    c = KINDS[kind](dv, 41)
    want = c()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [torch.full((c.need,), 255, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    outs = [c(stream=s, workspace=w) for _ in range(6) for s, w in zip(streams, ws)]
    outs += [c(stream=s.cuda_stream) for _ in range(2) for s in streams]     # workspaces of the call's own
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("kind", KINDS)
def test_captured_calls_read_their_inputs_anew(dv, kind):
    """Queries and lengths that change between replays; the workspace is the graph's."""
    c = KINDS[kind](dv, 51)
    q, lens = c.args[0], c.args[2]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c()
    for i in range(4):
        c.q = P.queries(q.shape[0], q.shape[1], q.shape[2], seed=60 + i)
        # not longer than the rows that are filled; every second one empty in one replay
        c.lens = [max(0, n - 31 * i) if not (i == 2 and j & 1) else 0 for j, n in enumerate(c.lens)]
        q.copy_(c.q)
        lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        g.replay()
        check(out, c.ref(), c.bound)


# --------------------------------------------------------------- largest counts ---
def some(c, at):
    """The plain result of sequences `at` alone."""
    lens = [c.lens[i] for i in at]
    if isinstance(c, Prefix):
        return P.attention(c.q[at], c.pool, c.table[at], lens, haze=c.haze, ptable=c.ptable, prefix=c.prefix)
    return P.attention(c.q[at], c.pool, c.table[at], lens, haze=c.haze)


def test_three_launches_over_4096_sequences(dv):
    c = Decode(dv, 2, 1, 64, [(i * 7) % 71 for i in range(4096)], seed=61)
    out = c()
    check(out, c.ref(), DECODE)
    assert (out[::71] == 0).all()


def test_prefix_read_once_by_4096_sequences_of_16_heads(dv):
    """65536 rows per KV head: 512 row tiles, more than the SMs; one split."""
    c = Prefix(dv, 16, 1, 64, [i % 3 for i in range(4096)], 130, 62, False)
    check(c(), c.ref(), PREFIX)


@pytest.mark.parametrize("split", [False, True])
def test_1024_kv_heads(dv, split):
    lens = [1, 0, 70]
    c = Prefix(dv, 1024, 1024, 64, lens, 140, 63, split)
    check(c(), c.ref(), PREFIX)
    d = Decode(dv, 1024, 1024, 64, lens, 64)
    check(d(), d.ref(), DECODE)


@pytest.mark.parametrize("prefix", [9000, 32768])
def test_one_split_of_a_long_prefix(dv, prefix):
    """So many rows that a CTA walks the whole prefix."""
    c = Prefix(dv, 7, 7, 128, [i % 2 for i in range(2500)], prefix, 65, False)
    at = [0, 1, 777, 1500, 2499]
    check(c()[at], some(c, at), PREFIX)


@pytest.mark.parametrize("d", [64, 256])
def test_append_and_read_over_4096_sequences(dv, d):
    B, H = 4096, 1
    g = torch.Generator().manual_seed(d)
    n = torch.randint(0, 4, (B,), generator=g)
    n[100], n[4095] = 300, 129
    start = torch.randint(0, 200, (B,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)])
    T, W = int(cu[-1]), 8
    table = torch.randperm(B * W, generator=g).to(torch.int32).reshape(B, W)
    pool = dict(k=torch.zeros((B * W, H, 64, d), dtype=torch.int8), v=torch.zeros((B * W, H, d, 64), dtype=torch.int8),
                ks=torch.zeros((B * W, H, 64), dtype=torch.bfloat16), vs=torch.zeros((B * W, H, 64), dtype=torch.bfloat16))
    k, v = (torch.randn((T, H, d), generator=g).to(torch.bfloat16) for _ in range(2))
    c = to_gpu(dv, pool, table)
    sg, cg = i32(start.tolist()), i32(cu.tolist())
    dv.dvssq_kv_append(c, k.cuda(), v.cuda(), sg, cg)
    b = torch.repeat_interleave(torch.arange(B), n)
    pos = start[b] + torch.arange(T) - cu[b]
    page, slot = table[b, pos // 64].long(), pos % 64
    kc, ks = P.hold(k)
    vc, vs = P.hold(v)
    pool["k"][page, :, slot], pool["ks"][page, :, slot] = kc, ks
    pool["v"][page, :, :, slot], pool["vs"][page, :, slot] = vc, vs
    assert torch.equal(c.k.cpu(), pool["k"]) and torch.equal(c.v.cpu(), pool["v"])
    assert torch.equal(c.k_scale.cpu(), pool["ks"]) and torch.equal(c.v_scale.cpu(), pool["vs"])
    ko, vo = dv.dvssq_kv_read(c, sg, cg, T)
    assert torch.equal(ko.cpu(), (kc.float() * ks.float()[..., None]).to(torch.bfloat16))
    assert torch.equal(vo.cpu(), (vc.float() * vs.float()[..., None]).to(torch.bfloat16))
