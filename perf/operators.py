"""The operators of the 8-bit KV cache and how their work is counted.

Four operators serve a decode loop whose KV cache is held in 8 bits (one BF16
scale per token and head, pages of 64 tokens):

  write    ``dvssq_kv_append`` quantises new K and V rows into the cache's pages,
           and ``dvssq_kv_read`` brings the same rows back as BF16
  read     ``dvssq_kv_read`` alone, on a filled cache
  attn     ``dvssq_bss_attention_q8``: KV-BSS decode attention over the cache
  step     a decode step: append one token per sequence, then attend
  prefix   ``dvssq_bss_attention_prefix``: the same attention for a batch whose
           sequences share a long prefix, which is read once for all of them

Layout of the cache (P pages of 64 tokens, H KV heads of d dimensions):
  k   int8 [P][H][64][d]     ks  bf16 [P][H][64]
  v   int8 [P][H][d][64]     vs  bf16 [P][H][64]
  table  int32 [B][W]: page of the 64-token block w of sequence b
A row x of d values is held as  s = bf16(max|x| / 127),  c = clip(rint(x / s), -127, 127)
(c = 0 where s = 0) and stands for c s.

Attention, for each query head h of KV head h // G over the L keys of its sequence:
  s_l = (q . k_l) tau / sqrt(d),  m = max_l s_l,  s_l < m - haze dropped (haze > 0),
  out = sum_l exp(s_l - m) v_l / sum_l exp(s_l - m);  zero where L = 0.
"""
import math
import random

import torch

own = False

PAGE = 64
TAU, HAZE = 1.10, 12.0
# (query heads, KV heads, head dimension)
SPARK, MINICPM = (16, 4, 256), (16, 2, 128)
HEADS = (SPARK, MINICPM, (8, 4, 256), (8, 2, 128), (6, 2, 128), (8, 8, 64), (20, 4, 64), (10, 2, 256))
DEV = "cuda"


def listed():
    return [
        # one decode step's new rows for a small batch: latency
        case("write", MINICPM, 16, 2048, new=1, name="write_decode_b16"),
        # the prompt of one sequence, page-aligned
        case("write", SPARK, 1, 4096, new=4096, name="write_prefill_4096"),
        # chunks of several prompts, each starting inside a page
        case("write", MINICPM, 7, 1100, new=777, name="write_ragged_b7"),
        # the last 512 tokens of each sequence, as a sliding-window layer wants them
        case("read", SPARK, 8, 6000, new=512, name="read_window_512_b8"),
        # whole contexts brought back, as a re-computation in BF16 wants them
        case("read", SPARK, 4, 8192, new=8192, name="read_context_8192_b4"),
        # a conversation's first tokens: latency
        case("attn", MINICPM, 1, 17, name="attn_17_b1"),
        # long contexts with flat attention: every key counts
        case("attn", SPARK, 4, 32768, bind=0, name="attn_32768_b4"),
        # a ragged batch whose binding keys leave most of the context below the haze floor
        case("attn", MINICPM, 32, 8000, name="attn_ragged_8000_b32"),
        # the decode step of a served batch
        case("step", SPARK, 16, 2048, bind=0, name="step_2048_b16"),
        # a short system prompt shared by a few sequences
        case("prefix", MINICPM, 4, 64, prefix=512, name="prefix_512_b4"),
        # odd sizes: three query heads per KV head, a prefix that ends inside a page
        case("prefix", (6, 2, 128), 24, 300, prefix=5001, bind=0, name="prefix_5001_b24"),
        # many samples of one long document
        case("prefix", SPARK, 64, 256, prefix=32768, bind=0, name="prefix_32768_b64"),
    ]


def case(kind, heads, batch, ctx, new=0, prefix=0, bind=2, haze=HAZE, name=None):
    """``ctx``: longest context of a sequence (its own part, where a prefix is shared); ``new``: rows
    written or read per sequence at most; ``bind``: binding keys planted per sequence and KV head."""
    hq, hkv, d = heads
    c = dict(kind=kind, hq=hq, hkv=hkv, d=d, batch=batch, ctx=ctx, new=new, prefix=prefix, bind=bind, haze=haze)
    return c if name is None else dict(c, name=name)


def draw(rng):
    log = lambda lo, hi: min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))  # noqa: E731
    kind = rng.choice(("write", "read", "attn", "attn", "step", "prefix", "prefix"))
    heads = rng.choice(HEADS)
    hq, hkv, d = heads
    batch = log(1, 64)
    bind = rng.choice((0, 1, 2, 4))
    haze = rng.choice((HAZE, HAZE, 0.0))
    if kind in ("write", "read"):
        most = max(1, min(8192, (2048 if kind == "write" else 6144) * 4 * 4 * 256 // (batch * hkv * d)))
        ctx = log(1, most)
        return case(kind, heads, batch, ctx, new=log(1, ctx), bind=0)
    if kind in ("attn", "step"):
        most = max(1, min(32768, 4 * 4 * 16384 * 256 // (batch * hkv * d)))
        return case(kind, heads, batch, log(1, most), new=1 if kind == "step" else 0, bind=bind, haze=haze)
    return case(kind, heads, batch, log(1, 256), prefix=log(64, 32768), bind=bind, haze=haze)


# ------------------------------------------------------------------ sizes ---
def sizes(c):
    """Lengths that go by the case alone: (lens, start, new), each a list of one number per sequence.
    ``lens``: tokens in the cache before the call; start, new: the rows written or read."""
    r = random.Random("%(kind)s %(hq)d %(hkv)d %(d)d %(batch)d %(ctx)d %(new)d %(prefix)d" % c)
    lens = [c["ctx"]] + [r.randint(max(0, c["ctx"] // 4), c["ctx"]) for _ in range(c["batch"] - 1)]
    if c["kind"] in ("attn", "prefix") and c["batch"] > 4:
        lens[1], lens[2] = 0, 1
    if c["kind"] == "step":
        lens = [max(0, n - 1) for n in lens]  # the new token brings them to ctx
        return lens, list(lens), [1] * c["batch"]
    if c["kind"] in ("write", "read"):
        new = [c["new"]] + [r.randint(max(1, c["new"] // 2), c["new"]) for _ in range(c["batch"] - 1)]
        lens = [max(n, k) for n, k in zip(lens, new)]
        return lens, [n - k for n, k in zip(lens, new)], new
    return lens, [0] * c["batch"], [0] * c["batch"]


def work(c):
    lens, _, new = sizes(c)
    hq, hkv, d, b = c["hq"], c["hkv"], c["d"], c["batch"]
    row = hkv * 2 * (d + 2)                    # codes and scales of one token's K and V
    if c["kind"] == "write":                   # BF16 in, codes and scales out and in again, BF16 out
        return {"bytes": sum(new) * (2 * hkv * 4 * d + 2 * row), "flops": sum(new) * hkv * d * 2 * 6}
    if c["kind"] == "read":
        return {"bytes": sum(new) * (hkv * 4 * d + row), "flops": sum(new) * hkv * d * 2}
    total = sum(lens) + sum(new) + c["prefix"]
    fl = 4 * hq * d * (sum(lens) + sum(new) + b * c["prefix"])
    return {"bytes": total * row + sum(new) * hkv * 4 * d + b * hq * 4 * d, "flops": fl}


# ----------------------------------------------------------------- inputs ---
def hold(x):
    """FP32 rows -> (codes as FP32 whole numbers, BF16 scales)."""
    s = (x.abs().amax(-1) / 127.0).to(torch.bfloat16)
    f = s.float().unsqueeze(-1)
    return torch.where(f > 0, (x / f).round().clamp(-127, 127), torch.zeros_like(x)), s


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    lens, start, new = sizes(c)
    hq, hkv, d, b = c["hq"], c["hkv"], c["d"], c["batch"]
    w = max(1, -(-max(n + (1 if c["kind"] == "step" else 0) for n in lens) // PAGE))
    pw = -(-c["prefix"] // PAGE)
    pages = b * w + pw + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    q = randn(b, hq, d).to(torch.bfloat16)
    st = dict(c, q=q, table=perm[: b * w].reshape(b, w).contiguous(), ptable=perm[b * w: b * w + pw].contiguous(),
              lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if c["kind"] != "write":
        # contexts: keys and values with a few strong channels, and planted binding keys whose
        # logit for the group's first head is near 16
        amp = 1.0 + 3.0 * (torch.rand(d, generator=g, device=DEV) < 0.03)
        k, v = randn(pages, hkv, PAGE, d) * (amp / amp.square().mean().sqrt()), randn(pages, hkv, PAGE, d)
        if c["bind"]:
            u = q[:, ::hq // hkv].float()
            u = u * (16.0 * math.sqrt(d) / TAU / u.square().sum(-1, keepdim=True))
            longest = max(n for n in lens) if not c["prefix"] else c["prefix"]
            for i in range(c["bind"]):
                at = (torch.rand(b, generator=g, device=DEV) * (st["lens"] if not c["prefix"] else longest)).long()
                page = st["ptable"].long()[at // PAGE] if c["prefix"] else st["table"].long()[torch.arange(b, device=DEV), at // PAGE]
                k[page, :, at % PAGE] = u + 0.05 * randn(b, hkv, d)
        kc, ks = hold(k.to(torch.bfloat16).float())
        vc, vs = hold(v.to(torch.bfloat16).float())
        st.update(k=kc.to(torch.int8), ks=ks, v=vc.to(torch.int8).transpose(2, 3).contiguous(), vs=vs)
    else:
        st.update(k=torch.zeros((pages, hkv, PAGE, d), dtype=torch.int8, device=DEV), ks=torch.zeros((pages, hkv, PAGE), dtype=torch.bfloat16, device=DEV),
                  v=torch.zeros((pages, hkv, d, PAGE), dtype=torch.int8, device=DEV), vs=torch.zeros((pages, hkv, PAGE), dtype=torch.bfloat16, device=DEV))
    if c["kind"] in ("write", "read", "step"):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        st["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        st["tokens"] = cu[-1]
        if c["kind"] != "read":
            # the new rows are slices of a fused projection's output [T][hq + 2 hkv][d]
            qkv = randn(cu[-1], hq + 2 * hkv, d).to(torch.bfloat16)
            st["new_k"], st["new_v"] = qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
        if c["kind"] == "step":
            st["lens"] = st["lens"] + 1
    return st


# -------------------------------------------------------------------- run ---
def run(st):
    return run_own(st) if own else run_plain(st)


def run_own(st):
    from mixed_precision_weight_b200 import binding as dv

    cache = dv.KvCache(st["k"], st["v"], st["ks"], st["vs"], st["table"])
    if st["kind"] == "write":
        dv.dvssq_kv_append(cache, st["new_k"], st["new_v"], st["start"], st["cu"])
        k, v = dv.dvssq_kv_read(cache, st["start"], st["cu"], st["tokens"])
        return {"k": k, "v": v, "ks": st["ks"], "vs": st["vs"]}
    if st["kind"] == "read":
        k, v = dv.dvssq_kv_read(cache, st["start"], st["cu"], st["tokens"])
        return {"k": k, "v": v}
    if st["kind"] == "step":
        dv.dvssq_kv_append(cache, st["new_k"], st["new_v"], st["start"])
    if st["kind"] == "prefix":
        return dv.dvssq_bss_attention_prefix(st["q"], cache, st["lens"], st["ptable"], st["prefix"], tau=TAU, haze=st["haze"], y_dtype=dv.Y_BF16)
    out = dv.dvssq_bss_attention_q8(st["q"], cache, st["lens"], tau=TAU, haze=st["haze"], y_dtype=dv.Y_BF16)
    return {"out": out, "ks": st["ks"], "vs": st["vs"]} if st["kind"] == "step" else out


def places(st):
    """(page, slot) of each row written or read."""
    t = torch.arange(st["tokens"], device=DEV)
    cu = st["cu"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = st["start"].long()[b] + t - cu[b]
    return st["table"].long()[b, pos // PAGE], pos % PAGE


def append_plain(st):
    page, slot = places(st)
    kc, ks = hold(st["new_k"].float())
    vc, vs = hold(st["new_v"].float())
    st["k"][page, :, slot] = kc.to(torch.int8)
    st["v"][page, :, :, slot] = vc.to(torch.int8)
    st["ks"][page, :, slot] = ks
    st["vs"][page, :, slot] = vs


def read_plain(st):
    page, slot = places(st)
    k = st["k"][page, :, slot].float() * st["ks"][page, :, slot].float().unsqueeze(-1)
    v = st["v"][page, :, :, slot].float() * st["vs"][page, :, slot].float().unsqueeze(-1)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def context(st, table):
    """K and V of whole pages in FP32: [...][H][W 64][d] for a table [...][W]."""
    t = table.long()
    k = st["k"][t].float() * st["ks"][t].float().unsqueeze(-1)
    v = st["v"][t].float() * st["vs"][t].float().unsqueeze(-2)
    k = k.transpose(-4, -3)
    v = v.transpose(-4, -3).transpose(-2, -1)
    return k.reshape(*k.shape[:-3], -1, k.shape[-1]), v.reshape(*v.shape[:-3], -1, v.shape[-1])


def run_plain(st):
    if st["kind"] == "write":
        append_plain(st)
        k, v = read_plain(st)
        return {"k": k, "v": v, "ks": st["ks"], "vs": st["vs"]}
    if st["kind"] == "read":
        k, v = read_plain(st)
        return {"k": k, "v": v}
    if st["kind"] == "step":
        append_plain(st)
    b, hq, d = st["q"].shape
    hkv = st["hkv"]
    q = st["q"].float().reshape(b, hkv, hq // hkv, d)
    k, v = context(st, st["table"])
    s = (q @ k.transpose(-1, -2)) * (TAU / math.sqrt(d))
    s = s.masked_fill(torch.arange(s.shape[-1], device=DEV) >= st["lens"].reshape(b, 1, 1, 1), -math.inf)
    if st["prefix"]:
        pk, pv = context(st, st["ptable"])
        n = st["prefix"]
        rows = q.transpose(0, 1).reshape(hkv, -1, d)
        sp = ((rows @ pk[:, :n].transpose(-1, -2)) * (TAU / math.sqrt(d))).reshape(hkv, b, hq // hkv, n).transpose(0, 1)
        s = torch.cat([sp, s], -1)
    m = s.amax(-1, keepdim=True)
    if st["haze"] > 0:
        s = s.masked_fill(s < m - st["haze"], -math.inf)
    p = torch.exp(s - m.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    if st["prefix"]:
        out = p[..., n:] @ v + (p[..., :n].transpose(0, 1).reshape(hkv, -1, n) @ pv[:, :n]).reshape(hkv, b, hq // hkv, d).transpose(0, 1)
    else:
        out = p @ v
    out = torch.where(total > 0, out / total, torch.zeros_like(out)).reshape(b, hq, d).to(torch.bfloat16)
    return {"out": out, "ks": st["ks"], "vs": st["vs"]} if st["kind"] == "step" else out


# ------------------------------------------------------------------ exact ---
def exact(c, seed):
    """What run() returns, from the definitions in 64 bits, one sequence and KV head after the other."""
    st = prepare(c, seed)
    lens, start, new = sizes(c)
    hq, hkv, d, b = c["hq"], c["hkv"], c["d"], c["batch"]
    table, cu = st["table"].tolist(), st["cu"].tolist() if "cu" in st else None

    def held(x):
        x = x.double()
        s = (x.abs().max(-1).values / 127).to(torch.bfloat16).double()
        code = torch.round(x / s.unsqueeze(-1)).clamp(-127, 127)
        return torch.where(s.unsqueeze(-1) > 0, code, 0.0), s

    def where_of(i):
        pos = torch.arange(start[i], start[i] + new[i], device=DEV)
        return st["table"][i].long()[pos // PAGE], pos % PAGE

    ks, vs = st["ks"].double(), st["vs"].double()
    kc, vc = st["k"].to(torch.int16), st["v"].to(torch.int16)
    if c["kind"] in ("write", "step"):
        kr, ksr = held(st["new_k"])
        vr, vsr = held(st["new_v"])
        for i in range(b):
            page, slot = where_of(i)
            a, z = cu[i], cu[i + 1]
            ks[page, :, slot], vs[page, :, slot] = ksr[a:z], vsr[a:z]
            kc[page, :, slot], vc[page, :, :, slot] = kr[a:z].to(torch.int16), vr[a:z].to(torch.int16)
    if c["kind"] in ("write", "read"):
        k = torch.empty((cu[-1], hkv, d), dtype=torch.float64, device=DEV)
        v = torch.empty_like(k)
        for i in range(b):
            page, slot = where_of(i)
            k[cu[i]: cu[i + 1]] = kc[page, :, slot].double() * ks[page, :, slot].unsqueeze(-1)
            v[cu[i]: cu[i + 1]] = vc[page, :, :, slot].double() * vs[page, :, slot].unsqueeze(-1)
        return {"k": k, "v": v, "ks": ks, "vs": vs} if c["kind"] == "write" else {"k": k, "v": v}

    def rows_of(pages, h, n):
        pages = torch.tensor(pages[: -(-n // PAGE)], dtype=torch.long, device=DEV)
        k = (kc[pages, h].double() * ks[pages, h].unsqueeze(-1)).reshape(-1, d)[:n]
        v = (vc[pages, h].double() * vs[pages, h].unsqueeze(-2)).transpose(1, 2).reshape(-1, d)[:n]
        return k, v

    out = torch.zeros((b, hq, d), dtype=torch.float64, device=DEV)
    g = hq // hkv
    for h in range(hkv):
        shared = rows_of(st["ptable"].tolist(), h, c["prefix"]) if c["prefix"] else None
        for i in range(b):
            k, v = rows_of(table[i], h, lens[i] + (1 if c["kind"] == "step" else 0))
            qi = st["q"][i, h * g: (h + 1) * g].double()
            s = qi @ k.T
            if shared is not None:
                s = torch.cat([qi @ shared[0].T, s], 1)
            if not s.shape[1]:
                continue
            s = s * (TAU / math.sqrt(d))
            m = s.max(1, keepdim=True).values
            p = torch.exp(s - m)
            if c["haze"] > 0:
                p = torch.where(s < m - c["haze"], 0.0, p)
            p = p / p.sum(1, keepdim=True)
            n = c["prefix"]
            out[i, h * g: (h + 1) * g] = p[:, n:] @ v + (p[:, :n] @ shared[1] if shared is not None else 0.0)
    return {"out": out, "ks": ks, "vs": vs} if c["kind"] == "step" else out
