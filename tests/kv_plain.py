"""Plain 64-bit implementation of the 8-bit KV cache and of KV-BSS attention over
it, and seeded caches for the tests.  CPU tensors throughout."""
import math

import torch

PAGE = 64


def hold(x):
    """BF16 rows [..., d] -> (codes int8 [..., d], scales bf16 [...]): the held form of the cache."""
    x = x.double()
    finite = torch.isfinite(x).all(-1)
    s = (x.abs().amax(-1) / 127.0).to(torch.float32).to(torch.bfloat16)
    sd = s.double().unsqueeze(-1)
    # the quotient of two 8-bit significands is a tie or at least 1/510 from one: fp64 decides it
    c = torch.where((sd > 0) & finite.unsqueeze(-1), torch.round(x / sd).clamp(-127, 127), torch.zeros_like(x))
    return c.to(torch.int8), torch.where(finite, s, torch.full_like(s, math.nan))


def places(table, start, cu):
    """[(sequence, row, page, slot)] of every row."""
    out = []
    for b in range(table.shape[0]):
        for i in range(int(cu[b + 1] - cu[b])):
            pos = int(start[b]) + i
            out.append((b, int(cu[b]) + i, int(table[b, pos // PAGE]), pos % PAGE))
    return out


def append(pool, table, k, v, start, cu):
    """Writes the held rows into pool = dict(k, v, ks, vs) in place."""
    kc, ks = hold(k)
    vc, vs = hold(v)
    for _, t, page, slot in places(table, start, cu):
        pool["k"][page, :, slot] = kc[t]
        pool["v"][page, :, :, slot] = vc[t]
        pool["ks"][page, :, slot] = ks[t]
        pool["vs"][page, :, slot] = vs[t]


def read(pool, table, start, cu, k_out, v_out):
    for _, t, page, slot in places(table, start, cu):
        # a 7-bit code times an 8-bit significand: exact in fp32, rounded once
        k_out[t] = (pool["k"][page, :, slot].float() * pool["ks"][page, :, slot].float()[:, None]).to(torch.bfloat16)
        v_out[t] = (pool["v"][page, :, :, slot].float() * pool["vs"][page, :, slot].float()[:, None]).to(torch.bfloat16)


def keys_values(pool, pages, n):
    """K and V [H][n][d] in fp64 of the first n tokens of a page list."""
    pages = [int(x) for x in pages[: -(-n // PAGE)]]
    k = pool["k"][pages].double() * pool["ks"][pages].double().unsqueeze(-1)      # [w][H][64][d]
    v = pool["v"][pages].double() * pool["vs"][pages].double().unsqueeze(-2)      # [w][H][d][64]
    H, d = k.shape[1], k.shape[3]
    return (k.transpose(0, 1).reshape(H, -1, d)[:, :n],
            v.permute(1, 0, 3, 2).reshape(H, -1, d)[:, :n])


def attention(q, pool, table, lens, tau=1.10, haze=12.0, ptable=None, prefix=0):
    """[B][Hq][d] in fp64; zeros where a sequence has no key."""
    B, Hq, d = q.shape
    H = pool["k"].shape[1]
    G = Hq // H
    out = torch.zeros((B, Hq, d), dtype=torch.float64)
    for b in range(B):
        k, v = keys_values(pool, table[b], int(lens[b]))
        if prefix:
            pk, pv = keys_values(pool, ptable, prefix)
            k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
        if k.shape[1] == 0:
            continue
        s = torch.einsum("hgd,hld->hgl", q[b].double().reshape(H, G, d), k) * (tau / math.sqrt(d))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        if haze > 0:
            p = torch.where(s < m - haze, torch.zeros_like(p), p)
        out[b] = (torch.einsum("hgl,hld->hgd", p, v) / p.sum(-1, keepdim=True)).reshape(Hq, d)
    return out


def filled(B, H, d, lens, seed, spare=3, prefix=0, bind=None, std=1.0):
    """A pool of random held rows with shuffled pages.  Slots that belong to no token, and pages that
    belong to no sequence, hold NaN scales and random codes; table entries past a sequence's
    pages hold nonsense.  ``bind`` = (queries [B][Hq][d], logit): one key per sequence (per KV head, for
    the group's first head) is planted with that logit."""
    g = torch.Generator().manual_seed(seed)
    W = max(1, max(-(-int(n) // PAGE) for n in lens)) + 1
    pw = -(-prefix // PAGE)
    need = sum(-(-int(n) // PAGE) for n in lens) + pw
    P = need + spare
    perm = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((B, W), 2 ** 31 - 1, dtype=torch.int32)
    used = torch.zeros((P, PAGE), dtype=torch.bool)
    at = pw
    ptable = perm[:pw].clone()
    for w in range(pw):
        used[int(ptable[w]), : min(PAGE, prefix - PAGE * w)] = True
    for b in range(B):
        n = int(lens[b])
        for w in range(-(-n // PAGE)):
            table[b, w] = perm[at]
            used[int(perm[at]), : min(PAGE, n - PAGE * w)] = True
            at += 1
    k = torch.randn((P, H, PAGE, d), generator=g) * std
    v = torch.randn((P, H, PAGE, d), generator=g)
    if bind is not None:
        q, logit = bind
        G = q.shape[1] // H
        u = q[:, ::G].float()
        u = u * (logit * math.sqrt(d) / 1.10 / u.square().sum(-1, keepdim=True))
        for b in range(B):
            n = prefix if prefix else int(lens[b])
            if n:
                i = int(torch.randint(n, (1,), generator=g))
                page = int(ptable[i // PAGE] if prefix else table[b, i // PAGE])
                k[page, :, i % PAGE] = u[b]
    kc, ks = hold(k.to(torch.bfloat16))
    vc, vs = hold(v.to(torch.bfloat16))
    dead = ~used[:, None, :].expand(P, H, PAGE)
    ks[dead], vs[dead] = math.nan, math.nan
    return dict(k=kc, v=vc.transpose(2, 3).contiguous(), ks=ks, vs=vs), table, ptable


def queries(B, Hq, d, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, Hq, d), generator=g).to(torch.bfloat16)
