"""Attention over keys that belong to more than one row set, as measured: cross attention (a
step's rows over all cached keys of another sequence, an encoder's states or a document), shared
attention (requests that continue one long prefix: the prefix is computed once for the rows of
all of them, each request's own keys apart, both joined), and the join itself (partial attention
results of the same queries over disjoint keys, by their log-sum-exp).

`run` computes an operator in plain torch operations, or (own = True) calls the framework.

The cache: pages of `ps` tokens, per page and KV head a block [ps, hd].  bf16 values, or 4-bit
values: e2m1 codes (two to a byte, the even dim in the low nibble) and one e4m3 scale per 16
dims; a value is code * scale * the tensor's global factor.  Token t of sequence b sits in page
table[b, t / ps], row t % ps.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def listed():
    gqa = dict(Hq=32, Hkv=8, hd=128)
    return [
        # one token of one decoder over 1500 encoder states: latency
        dict(name="cross_step_b1", op="cross", B=1, rlo=1, R=1, lo=1500, hi=1500, ps=64, kind="bf16", **gqa),
        # one token of 32 decoders with a KV head for each query head, over ragged states: bytes
        dict(name="cross_step_b32_hd64", op="cross", B=32, rlo=1, R=1, lo=300, hi=3000, ps=32, kind="bf16", Hq=16, Hkv=16, hd=64),
        # one token of 48 requests over long documents cached in 4 bits: bytes
        dict(name="cross_step_b48_f4", op="cross", B=48, rlo=1, R=1, lo=1000, hi=16000, ps=64, kind="f4", **gqa),
        # the rows of 8 draft trees over the 4-bit states of images
        dict(name="cross_tree_b8_f4", op="cross", B=8, rlo=37, R=61, lo=577, hi=4097, ps=32, kind="f4", **gqa),
        # two prompts over long encoder states: the products
        dict(name="cross_prompt", op="cross", B=2, rlo=2047, R=2047, lo=4099, hi=4099, ps=64, kind="bf16", **gqa),
        # one token of two samples of a short prompt: latency
        dict(name="shared_step_b2", op="shared", groups=1, B=2, rlo=1, R=1, lo=5, hi=40, plo=700, phi=700, tree=False, ps=64, kind="bf16", tail="bf16", **gqa),
        # one token of 32 samples of one prompt: the prompt's bytes once
        dict(name="shared_step_b32", op="shared", groups=1, B=32, rlo=1, R=1, lo=1, hi=1024, plo=8192, phi=8192, tree=False, ps=64, kind="bf16", tail="bf16", **gqa),
        # one token of 64 requests on four documents in 4 bits, their own keys in bf16
        dict(name="shared_step_b64_f4", op="shared", groups=4, B=64, rlo=1, R=1, lo=16, hi=500, plo=8000, phi=32000, tree=False, ps=64, kind="f4", tail="bf16", **gqa),
        # the verification of 32 samples' 61-slot trees behind one prompt
        dict(name="shared_tree_b32", op="shared", groups=1, B=32, rlo=61, R=61, lo=64, hi=700, plo=8192, phi=8192, tree=True, ps=64, kind="bf16", tail="bf16", **gqa),
        # four users' prompts behind one long system prompt in 4 bits, causal
        dict(name="shared_chunk_f4", op="shared", groups=1, B=4, rlo=301, R=509, lo=0, hi=0, plo=16001, phi=16001, tree=False, ps=128, kind="f4", tail="f4", **gqa),
        # a step whose keys lie in two caches: latency
        dict(name="merge_step", op="merge", parts=2, N=8, H=32, hd=128, dtype="bf16", out="bf16"),
        # a long prompt whose keys were taken in four segments
        dict(name="merge_prompt", op="merge", parts=4, N=8191, H=32, hd=128, dtype="f32", out="bf16"),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["cross", "cross", "shared", "shared", "merge"])
        if op == "merge":
            c = dict(op=op, parts=rng.randint(1, 8), N=logint(1, 9000), H=rng.choice([1, 5, 8, 28, 32, 64]), hd=rng.choice([64, 80, 128, 256]))
            c["dtype"], c["out"] = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"])
        else:
            c = dict(op=op, hd=rng.choice([64, 128]), ps=rng.choice([16, 32, 64, 128]), kind=rng.choice(["bf16", "f4"]), Hkv=rng.choice([1, 2, 4, 8, 16]))
            c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 7, 8])
            c["B"] = logint(1, 64)
            c["R"] = rng.choice([1, 1, logint(1, 64), logint(1, 2000)])
            c["rlo"] = rng.choice([1, c["R"]])
        if op == "cross":
            c["lo"] = rng.choice([0, 1, logint(1, 4000)])
            c["hi"] = c["lo"] + logint(1, 16000)
        if op == "shared":
            c["groups"] = rng.randint(1, min(6, c["B"]))
            c["tree"] = c["R"] <= 64 and rng.random() < 0.6
            c["tail"] = rng.choice(["bf16", "f4"])
            c["lo"] = rng.choice([0, logint(1, 500)])
            c["hi"] = c["lo"] + logint(1, 1500)
            c["plo"] = rng.choice([0, 1, logint(1, 8000)])
            c["phi"] = c["plo"] + logint(1, 32000)
        same = [work(d) for d in listed() if d["op"] == op]
        w = work(c)
        if all(w[k] <= max(x[k] for x in same) for k in w) and _scores(c) < 1.2e9:
            return c


def _spread(n, lo, hi, salt):
    """n numbers over [lo, hi] in an irregular order."""
    return [lo + (b * 2654435761 + salt) % (hi - lo + 1) if n > 1 else hi for b in range(n)]


def _ctx(case):
    """Keys of each sequence (cross), or each request's own keys before the step (shared)."""
    return _spread(case["B"], case["lo"], case["hi"], 12345)


def _rows(case):
    return _spread(case["B"], case["rlo"], case["R"], 777)


def _prefix(case):
    return _spread(case["groups"], case["plo"], case["phi"], 4242)


def _cu_groups(case):
    return [case["B"] * g // case["groups"] for g in range(case["groups"] + 1)]


def _group_rows(case):
    rows, at = _rows(case), _cu_groups(case)
    return [sum(rows[at[g]:at[g + 1]]) for g in range(case["groups"])]


def _scores(case):
    """Scores that the plain form holds at once."""
    if case["op"] == "merge":
        return 0
    pre = case["groups"] * max(_group_rows(case)) * max(_prefix(case)) if case["op"] == "shared" else 0
    rows = max(_rows(case))
    return case["Hq"] * max(pre, case["B"] * rows * (max(_ctx(case)) + rows))


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "merge":
        P, N, H, hd = case["parts"], case["N"], case["H"], case["hd"]
        st["outs"] = [torch.randn(N, H, hd, generator=g, device="cuda").to(_TYPE[case["dtype"]]) for _ in range(P)]
        st["lses"] = [2.0 * torch.randn(N, H, generator=g, device="cuda") + 6.0 for _ in range(P)]
        return st
    rows, ctx = _rows(case), _ctx(case)
    N = sum(rows)
    st["cu_rows"], st["lens"] = _cu(rows), torch.tensor(ctx, dtype=torch.int32, device="cuda")
    st["max_rows"] = max(rows)
    st["q"] = torch.randn(N, case["Hq"], case["hd"], generator=g, device="cuda", dtype=torch.bfloat16)
    spread = torch.exp(0.5 * torch.randn(case["Hkv"], 1, case["hd"], generator=g, device="cuda"))   # some key channels are large
    if op == "cross":
        st["cache"], st["max_len"] = _pool(case, ctx, case["kind"], spread, g), max(max(ctx), 1)
        return st
    pre = _prefix(case)
    st["prefix"] = _pool(case, pre, case["kind"], spread, g)
    st["prefix_lens"], st["max_prefix"] = torch.tensor(pre, dtype=torch.int32, device="cuda"), max(max(pre), 1)
    at = _cu_groups(case)
    st["cu_groups"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    st["max_group_rows"] = max(_group_rows(case))
    st["cu_group_rows"] = st["cu_rows"][st["cu_groups"].long()].contiguous()
    held = [n + r for n, r in zip(ctx, rows)]
    st["cache"], st["max_len"] = _pool(case, held, case["tail"], spread, g), max(held)
    st["mask"] = None
    if case["tree"]:   # ancestor-or-self masks of random trees whose parents precede their children
        B, R = case["B"], max(rows)
        parent = (torch.rand(B, R, generator=g, device="cuda") * torch.arange(R, device="cuda")).long()
        m = torch.eye(R, dtype=torch.uint8, device="cuda").repeat(B, 1, 1)
        for i in range(1, R):
            m[:, i] |= m[torch.arange(B, device="cuda"), parent[:, i].clamp(max=i - 1)]
        st["mask"] = m
    return st


_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pool(case, held, kind, spread, g):
    """Pages for held[b] tokens of each sequence in a shuffled pool with some spare pages."""
    Hkv, hd, ps = case["Hkv"], case["hd"], case["ps"]
    need = [(n + ps - 1) // ps for n in held]
    width, pages = max(max(need), 1), sum(need) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    have = slot < torch.tensor(need, device="cuda")[:, None]
    p = {"ps": ps, "kg": 1.0, "vg": 1.0}
    p["table"] = torch.where(have, perm[(at[:, None] + slot).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    k = torch.randn(pages, Hkv, ps, hd, generator=g, device="cuda", dtype=torch.bfloat16) * spread.to(torch.bfloat16)
    v = torch.randn(pages, Hkv, ps, hd, generator=g, device="cuda", dtype=torch.bfloat16)
    if kind == "f4":
        p["vg"] = 0.25
        (p["k"], p["ks"]), (p["v"], p["vs"]) = _quantise(k, p["kg"]), _quantise(v, p["vg"])
    else:
        p["k"], p["v"], p["ks"], p["vs"] = k, v, None, None
    if own:   # the handle that a user's program keeps
        from eagle_speculative_decoding_03_gb300 import binding as eb
        p["handle"] = eb.KVCache(p["k"], p["v"], p["table"], p["ks"], p["vs"], p["kg"], p["vg"])
    return p


def _quantise(x, glob):
    """bf16 values [..., hd] -> e2m1 codes [..., hd / 2] and e4m3 scales [..., hd / 16]."""
    y = x.float().unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / (6.0 * glob)).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = scale.float()[..., None] * glob
    mag = torch.where(unit > 0, y.abs() / unit, 0.0)
    code = torch.bucketize(mag, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)).to(torch.uint8)
    code = (code + 8 * (y < 0)).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8).contiguous(), scale.view(torch.uint8).contiguous()


def _cu(ns):
    return torch.tensor([sum(ns[:b]) for b in range(len(ns) + 1)], dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------------- plain forms
def _values(code, scale, glob):
    """The fp32 values that codes and scales stand for."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=code.device)
    nib = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    unit = scale.view(torch.float8_e4m3fn).float() * glob
    return (lut[nib.int()].unflatten(-1, (-1, 16)) * unit[..., None]).flatten(-2)


def _keys(p, length):
    """fp32 keys and values [B, length, Hkv, hd] of every sequence (anything behind its last key)."""
    t = torch.arange(length, device="cuda")
    page = p["table"].long()[:, t // p["ps"]].clamp(min=0)
    row = (t % p["ps"]).expand(page.shape)
    if p["ks"] is None:
        return p["k"][page, :, row].float(), p["v"][page, :, row].float()
    return _values(p["k"][page, :, row], p["ks"][page, :, row], p["kg"]), _values(p["v"][page, :, row], p["vs"][page, :, row], p["vg"])


def _part(q, cu, R, K, V, see):
    """Rows [N, Hq, hd] over their sequences' keys [B, L, Hkv, hd]: fp32 output and log-sum-exp.
    Sequence b's rows cu[b] .. cu[b + 1] are padded to R; see [B, R or 1, L]: which keys row i sees."""
    N, Hq, hd = q.shape
    B, L, Hkv, _ = K.shape
    cu = cu.long()
    i = torch.arange(R, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=N - 1)                              # [B, R] the rows
    x = q.float()[at].unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)     # [B, Hkv, G R, hd]
    s = torch.matmul(x, K.permute(0, 2, 3, 1)).unflatten(2, (-1, R)) / math.sqrt(hd)
    s = s.masked_fill(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.clamp(min=-1e30))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), V.transpose(1, 2)).unflatten(2, (-1, R)) / torch.where(z > 0, z, 1.0)
    lse = (top + z.log())[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)   # [B, R, Hq, hd]
    n = torch.arange(N, device="cuda")
    b = torch.searchsorted(cu, n, right=True) - 1
    return o[b, n - cu[b]], lse[b, n - cu[b]]


def _join(outs, lses):
    """Results over disjoint keys, joined: fp32 [N, H, hd] and [N, H]."""
    l = torch.stack(lses)
    top = l.amax(0).clamp(min=-1e30)
    w = torch.exp(l - top)
    z = w.sum(0)
    o = (torch.stack([x.float() for x in outs]) * w[..., None]).sum(0) / torch.where(z > 0, z, 1.0)[..., None]
    return o, top + z.log()


def _first(lens, L):
    return (torch.arange(L, device="cuda")[None, :] < lens.long()[:, None])[:, None]


def run(st):
    case, op = st["case"], st["op"]
    if own:
        return _run_own(st)
    if op == "merge":
        o, l = _join(st["outs"], st["lses"])
        return o.to(_TYPE[case["out"]]), l
    if op == "cross":
        L = st["max_len"]
        o, l = _part(st["q"], st["cu_rows"], st["max_rows"], *_keys(st["cache"], L), _first(st["lens"], L))
        return o.to(torch.bfloat16), l
    P, L, R = st["max_prefix"], st["max_len"], st["max_rows"]
    pre = _part(st["q"], st["cu_group_rows"], st["max_group_rows"], *_keys(st["prefix"], P), _first(st["prefix_lens"], P))
    i = torch.arange(R, device="cuda")
    j = torch.arange(L, device="cuda")[None, :] - st["lens"].long()[:, None]       # [B, L]: which of the step's rows
    see = j[:, None, :] <= i[None, :, None]                                # causal
    if st["mask"] is not None:
        m = torch.gather(st["mask"].bool(), 2, j.clamp(0, R - 1)[:, None, :].expand(-1, R, L))
        see = (j[:, None, :] < 0) | (m & (j[:, None, :] < R))
    tail = _part(st["q"], st["cu_rows"], R, *_keys(st["cache"], L), see)
    o, l = _join([pre[0], tail[0]], [pre[1], tail[1]])
    return o.to(torch.bfloat16), l


def _run_own(st):
    from eagle_speculative_decoding_03_gb300 import binding as eb
    case, op = st["case"], st["op"]
    if op == "merge":
        return eb.attention_merge(st["outs"], st["lses"], dtype=_TYPE[case["out"]], lse=True)
    if op == "cross":
        return eb.kv_cross_attention(st["cache"]["handle"], st["q"], st["cu_rows"], st["lens"], max_rows=st["max_rows"],
                                     max_len=st["max_len"], lse=True)
    return eb.kv_shared_attention(st["prefix"]["handle"], st["cu_groups"], st["prefix_lens"], st["cache"]["handle"], st["q"],
                                  st["cu_rows"], st["lens"], max_group_rows=st["max_group_rows"], max_prefix=st["max_prefix"],
                                  max_rows=st["max_rows"], max_len=st["max_len"], mask=st["mask"], lse=True)


# ------------------------------------------------------------------- work and exact values
def work(case):
    if case["op"] == "merge":
        e, s = case["N"] * case["H"], {"bf16": 2, "f32": 4}
        return {"bytes": e * (case["parts"] * (case["hd"] * s[case["dtype"]] + 4) + case["hd"] * s[case["out"]] + 4),
                "flops": 2 * e * case["parts"] * case["hd"]}
    Hkv, Hq, hd = case["Hkv"], case["Hq"], case["hd"]
    per = {"bf16": 4 * Hkv * hd, "f4": Hkv * (hd + hd // 8)}               # a token's key and value
    rows, ctx = _rows(case), _ctx(case)
    out = sum(rows) * Hq * (4 * hd + 4)
    if case["op"] == "cross":
        return {"bytes": sum(n for n, r in zip(ctx, rows) if r) * per[case["kind"]] + out,
                "flops": 4 * hd * Hq * sum(r * n for r, n in zip(rows, ctx))}
    pre = _prefix(case)
    seen = sum(r * n for r, n in zip(_group_rows(case), pre)) + sum(r * n + r * (r + 1) // 2 for r, n in zip(rows, ctx))   # (a tree's rows see no more)
    return {"bytes": sum(pre) * per[case["kind"]] + sum(n + r for n, r in zip(ctx, rows)) * per[case["tail"]] + out
            + (sum(r * r for r in rows) if case["tree"] else 0),
            "flops": 4 * hd * Hq * seen}


def exact(case, seed):
    """The operators from their definitions in 64 bits, request by request: shared attention is
    one softmax over the prefix's keys and the request's own."""
    st = prepare(case, seed)
    if case["op"] == "merge":
        w = [l.double().exp() for l in st["lses"]]
        return sum(o.double() * x[..., None] for o, x in zip(st["outs"], w)) / sum(w)[..., None], sum(w).log()
    if work(case)["flops"] > 1.2e12:
        return None
    Hq, Hkv, hd, ps = case["Hq"], case["Hkv"], case["hd"], case["ps"]
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def held(p, b, n, name):
        """Sequence b's first n keys or values, [n, Hkv, hd]."""
        pages = p["table"][b, :(n + ps - 1) // ps].long()

        def rows(x):
            return x[pages].transpose(1, 2).flatten(0, 1)[:n]
        c = rows(p[name])
        if p[name + "s"] is None:
            return c.double()
        c = c.int()
        mag = torch.empty(c.shape[:-1] + (hd,), dtype=torch.float64, device="cuda")
        mag[..., 0::2] = grid[(c & 7).long()] * (1 - 2 * ((c >> 3) & 1))
        mag[..., 1::2] = grid[((c >> 4) & 7).long()] * (1 - 2 * (c >> 7))
        return mag * (rows(p[name + "s"]).view(torch.float8_e4m3fn).double() * p[name + "g"]).repeat_interleave(16, -1)

    rows, ctx = _rows(case), _ctx(case)
    out = torch.zeros(sum(rows), Hq, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(rows), Hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, r) in enumerate(zip(ctx, rows)):
        if case["op"] == "cross":
            K, V = held(st["cache"], b, n, "k"), held(st["cache"], b, n, "v")
            sees = torch.ones(r, n, dtype=torch.bool, device="cuda")
        else:
            grp = sum(x <= b for x in _cu_groups(case)) - 1
            m = _prefix(case)[grp]
            K, V = (torch.cat([held(st["prefix"], grp, m, x), held(st["cache"], b, n + r, x)]) for x in ("k", "v"))
            sees = torch.ones(r, m + n + r, dtype=torch.bool, device="cuda")
            sees[:, m + n:] = st["mask"][b, :r, :r].bool() if case["tree"] else torch.ones(r, r, device="cuda").tril().bool()
        for h in range(Hq if r and K.shape[0] else 0):
            s = (st["q"][at:at + r, h].double() @ K[:, h // (Hq // Hkv)].T) * hd ** -0.5
            s[~sees] = -math.inf
            l = torch.logsumexp(s, 1)
            out[at:at + r, h], lse[at:at + r, h] = torch.exp(s - l[:, None]) @ V[:, h // (Hq // Hkv)], l
        at += r
    return out, lse
