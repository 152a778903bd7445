"""The cache operators of speculative decoding, as measured: rotary positions, appending
rotated keys and values to a paged cache (bf16 or 4-bit), tree / causal attention over that
cache, gathering it into the packed form the draft and verification steps read, and keeping
the accepted path of a verified tree.

`run` computes an operator in plain torch operations, or (own = True) calls the framework.

The cache: pages of `ps` tokens, per page and KV head a block [ps, hd].  bf16 values, or 4-bit
values: e2m1 codes (two to a byte, the even dim in the low nibble) and one e4m3 scale per 16
dims; a value is code * scale * the tensor's global factor.  Request b's token t sits in page
table[b, t / ps], row t % ps.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def listed():
    head = dict(Hq=32, Hkv=8, hd=128)
    rot = dict(rot=128, theta=5e5, inter=False, far=0)
    return [
        # the queries of 8 requests' next token at positions of a long conversation
        dict(name="rotary_step", op="rotary", N=8, H=32, hd=128, dtype="bf16", rot=128, theta=5e5, inter=False, far=100000),
        # a prompt's fp32 queries, half of each head rotated in adjacent pairs, far positions
        dict(name="rotary_prompt", op="rotary", N=8191, H=64, hd=128, dtype="f32", rot=64, theta=1e4, inter=True, far=1000000),
        # one new token of 32 requests: queries rotated, keys rotated into the pages, values stored
        dict(name="append_step", op="append", B=32, R=1, lo=256, hi=2048, ps=64, kind="bf16", **head, **rot),
        # four prompts into an empty 4-bit cache, then gathered back
        dict(name="append_prompt_f4", op="append", B=4, R=2047, lo=0, hi=0, ps=64, kind="f4", **head, **rot),
        # the draft's 2048-token prefix from bf16 pages to the packed cache
        dict(name="gather_b1", op="gather", B=1, lo=2048, hi=2048, ps=16, kind="bf16", Hkv=8, hd=128),
        # 32 ragged prefixes out of 4-bit pages
        dict(name="gather_b32_f4", op="gather", B=32, lo=256, hi=4096, ps=32, kind="f4", Hkv=8, hd=128),
        # one token of one request over a 2048-token cache: latency
        dict(name="attention_step_b1", op="attention", B=1, R=1, lo=2048, hi=2048, ps=64, kind="bf16", tree=False, **head),
        # one token of 32 requests over long ragged 4-bit caches: bytes
        dict(name="attention_step_b32_f4", op="attention", B=32, R=1, lo=2048, hi=32768, ps=64, kind="f4", tree=False, **head),
        # the verification of 61-slot trees, 8 requests of 4096 tokens, the 64-query-head target
        dict(name="attention_tree_b8", op="attention", B=8, R=61, lo=4096, hi=4096, ps=64, kind="bf16", tree=True, Hq=64, Hkv=8, hd=128),
        # a 509-token chunk of a prompt behind 32000 cached 4-bit tokens, causal
        dict(name="attention_chunk_f4", op="attention", B=1, R=509, lo=32000, hi=32000, ps=128, kind="f4", tree=False, **head),
        # the accepted path of one tree in one layer's cache: latency
        dict(name="accept_b1", op="accept", B=1, S=61, L=1, lo=2048, hi=2048, ps=64, Hkv=8, hd=128),
        # 32 trees of 49 slots in 16 layers' caches
        dict(name="accept_b32", op="accept", B=32, S=49, L=16, lo=64, hi=700, ps=64, Hkv=8, hd=128),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["rotary", "append", "gather", "attention", "attention", "accept"])
        hd, kind = rng.choice([64, 128]), rng.choice(["bf16", "f4"])
        c = dict(op=op, hd=hd, ps=rng.choice([16, 32, 64, 128]), kind=kind, Hkv=rng.choice([1, 2, 4, 8]))
        c["rot"] = rng.choice([hd, hd // 2, 16 * rng.randint(1, hd // 16)])
        c["theta"], c["inter"], c["far"] = rng.choice([1e4, 5e5]), rng.random() < 0.5, logint(1, 1000000)
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 7, 8])
        c["B"] = logint(1, 48)
        c["lo"] = logint(1, 2000)
        c["hi"] = c["lo"] + logint(1, 6000)
        if op == "rotary":
            c = {k: c[k] for k in ("op", "hd", "rot", "theta", "inter", "far")}
            c.update(N=logint(1, 8000), H=rng.choice([1, 5, 8, 28, 32, 40, 64]), dtype=rng.choice(["bf16", "f32"]))
        elif op == "append":
            if kind == "f4":
                c["lo"] = c["hi"] = 0
            c["R"] = logint(1, 64 if kind == "bf16" else 2000)
        elif op == "attention":
            c["tree"] = rng.random() < 0.4
            c["R"] = logint(1, 64) if c["tree"] else rng.choice([1, 1, logint(1, 300)])
            if rng.random() < 0.2:
                c["B"], c["lo"], c["hi"] = rng.choice([1, 2]), 1, logint(4000, 100000)
                c["lo"] = c["hi"] // 2
        elif op == "accept":
            c["S"], c["L"], c["kind"] = rng.randint(2, 64), logint(1, 16), "bf16"
            c["hi"] = c["lo"] + logint(1, 600)
        same = [work(d) for d in listed() if d["op"] == op]
        w = work(c)
        if all(w[k] <= max(x[k] for x in same) for k in w) and _pool_tokens(c) * c.get("Hkv", 1) * c.get("L", 1) <= 5000000:
            return c


def _ctx(case):
    """Cached keys of each request: spread over [lo, hi] in an irregular order."""
    lo, hi = case["lo"], case["hi"]
    return [lo + (b * 2654435761 + 12345) % (hi - lo + 1) if case["B"] > 1 else hi for b in range(case["B"])]


def _rows(case):
    return case.get("R", case.get("S", 0))


def _pool_tokens(case):
    return sum(n + _rows(case) for n in _ctx(case)) if "B" in case else 0


def _dst_span(case):
    """Accepted tokens of each request's tree: their slots lie behind the places they move to."""
    return [(b * 7 + 3) % (case["S"] // 2 + 1) if case["S"] > 2 else 0 for b in range(case["B"])]


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "rotary":
        N, H, hd = case["N"], case["H"], case["hd"]
        x = torch.randn(N, H, hd, generator=g, device="cuda")
        st["x"] = x.to(_TYPE[case["dtype"]])
        st["positions"] = torch.randint(0, case["far"] + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
        _rope(st, case)
        return st
    B, Hkv, hd, ps, R = case["B"], case["Hkv"], case["hd"], case["ps"], _rows(case)
    ctx = _ctx(case)
    kind = case.get("kind", "bf16")
    # pages of every request in a shuffled pool with some spare pages
    need = [(n + R + ps - 1) // ps for n in ctx]
    width, pages = max(max(need), 1), sum(need) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([sum(need[:b]) for b in range(B)], device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    have = slot < torch.tensor(need, device="cuda")[:, None]
    st["table"] = torch.where(have, perm[(at[:, None] + slot).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    st["lens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    st["cu_rows"] = torch.arange(B + 1, device="cuda", dtype=torch.int32) * R
    layers = (case["L"],) if op == "accept" else ()
    spread = torch.exp(0.5 * torch.randn(Hkv, 1, hd, generator=g, device="cuda"))   # some key channels are large

    def pool(chan):
        shape = layers + (pages, Hkv, ps, hd)
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * chan.to(torch.bfloat16))

    if kind == "f4" and op == "append":
        st["k"] = torch.zeros(pages, Hkv, ps, hd // 2, dtype=torch.uint8, device="cuda")
        st["v"] = torch.zeros_like(st["k"])
        st["k_scale"] = torch.zeros(pages, Hkv, ps, hd // 16, dtype=torch.uint8, device="cuda")
        st["v_scale"] = torch.zeros_like(st["k_scale"])
    elif kind == "f4":
        st["k"], st["k_scale"] = _quantise(pool(spread), 1.0)
        st["v"], st["v_scale"] = _quantise(pool(torch.ones_like(spread)), 0.25)
    else:
        st["k"], st["v"] = pool(spread), pool(torch.ones_like(spread))
    st["k_global"], st["v_global"] = (1.0, 0.25) if kind == "f4" else (1.0, 1.0)
    N = B * R
    if op == "append":
        # the slices of one projection's output [queries | keys | values]
        Hq = case["Hq"]
        qkv = torch.randn(N, (Hq + 2 * Hkv) * hd, generator=g, device="cuda", dtype=torch.bfloat16)
        st["q_rows"] = qkv[:, :Hq * hd].unflatten(1, (Hq, hd))
        st["k_rows"] = qkv[:, Hq * hd:(Hq + Hkv) * hd].unflatten(1, (Hkv, hd))
        st["v_rows"] = qkv[:, (Hq + Hkv) * hd:].unflatten(1, (Hkv, hd))
        st["positions"] = (st["lens"][:, None] + torch.arange(R, device="cuda", dtype=torch.int32)).reshape(N).contiguous()
        st["cu_seqlens"] = _cu([n + R for n in ctx])
        st["total"] = sum(ctx) + N
        _rope(st, case)
    elif op == "gather":
        st["cu_seqlens"], st["total"] = _cu(ctx), sum(ctx)
    elif op == "attention":
        st["q"] = torch.randn(N, case["Hq"], hd, generator=g, device="cuda", dtype=torch.bfloat16)
        st["max_len"] = max(ctx) + R
        st["mask"] = None
        if case["tree"]:   # ancestor-or-self masks of random trees whose parents precede their children
            parent = (torch.rand(B, R, generator=g, device="cuda") * torch.arange(R, device="cuda")).long()
            m = torch.eye(R, dtype=torch.uint8, device="cuda").repeat(B, 1, 1)
            for i in range(1, R):
                m[:, i] |= m[torch.arange(B, device="cuda"), parent[:, i].clamp(max=i - 1)]
            st["mask"] = m
    elif op == "accept":
        S, span = case["S"], _dst_span(case)
        score = torch.rand(B, S, generator=g, device="cuda")
        n = torch.tensor(span, device="cuda")
        col = torch.arange(S, device="cuda")[None, :]
        score = torch.where(col > n[:, None], score, 2.0)
        pick = score.argsort(dim=1)                              # random slots behind the first n + 1
        pick = torch.where(col < n[:, None], pick, S).sort(dim=1).values
        st["accept_slots"] = torch.where(col < n[:, None], pick, -1).to(torch.int32).contiguous()
        st["accept_len"] = n.to(torch.int32)
    if own:   # the handle that a user's program keeps
        from eagle_speculative_decoding_03_gb300 import binding as eb
        per = [()] if not layers else [(i,) for i in range(case["L"])]
        caches = [eb.KVCache(st["k"][i], st["v"][i], st["table"], st["k_scale"][i] if kind == "f4" else None,
                             st["v_scale"][i] if kind == "f4" else None, st["k_global"], st["v_global"]) for i in per]
        st["cache"] = caches if layers else caches[0]
    return st


_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rope(st, case):
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
    st["inv_freq"] = case["theta"] ** (-i / case["rot"])
    if own:
        from eagle_speculative_decoding_03_gb300 import binding as eb
        st["rope"] = eb.Rope(case["rot"], theta=case["theta"], interleaved=case["inter"])


def _cu(ns):
    return torch.tensor([sum(ns[:b]) for b in range(len(ns) + 1)], dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------------- plain forms
def _quantise(x, glob):
    """bf16 values [..., hd] -> e2m1 codes [..., hd / 2] and e4m3 scales [..., hd / 16]."""
    y = x.float().unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / (6.0 * glob)).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = scale.float()[..., None] * glob
    mag = torch.where(unit > 0, y.abs() / unit, 0.0)
    # round to nearest, ties to the even code: the borders between neighbouring magnitudes
    code = ((mag > 0.25).to(torch.uint8) + (mag >= 0.75) + (mag > 1.25) + (mag >= 1.75) + (mag > 2.5) + (mag >= 3.5)
            + (mag > 5.0))
    code = (code + 8 * (y < 0)).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8).contiguous(), scale.view(torch.uint8).contiguous()


def _values(code, scale, glob):
    """The fp32 values that codes and scales stand for."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=code.device)
    nib = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    unit = scale.view(torch.float8_e4m3fn).float() * glob
    return (lut[nib.int()].unflatten(-1, (-1, 16)) * unit[..., None]).flatten(-2)


def _rotate(x, positions, inv_freq, inter):
    """fp32 rows [N, H, hd] rotated at their positions (angles in 64 bits)."""
    ang = positions.double()[:, None] * inv_freq
    c, s = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    rot = 2 * inv_freq.numel()
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _place(st, R):
    """Page and row of each request's R rows behind its cached keys."""
    ps = st["case"]["ps"]
    t = st["lens"].long()[:, None] + torch.arange(R, device="cuda")
    return torch.gather(st["table"].long(), 1, t // ps).reshape(-1), (t % ps).reshape(-1)


def _packed(st):
    """The cached keys and values of every request, packed [total, Hkv, hd] in bf16."""
    cu, ps = st["cu_seqlens"].long(), st["case"]["ps"]
    t = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    t = t - cu[b]
    page, row = st["table"].long()[b, t // ps], t % ps
    if "k_scale" not in st:
        return st["k"][page, :, row], st["v"][page, :, row]
    return (_values(st["k"][page, :, row], st["k_scale"][page, :, row], st["k_global"]).to(torch.bfloat16),
            _values(st["v"][page, :, row], st["v_scale"][page, :, row], st["v_global"]).to(torch.bfloat16))


def _attend(st):
    case = st["case"]
    B, R, Hkv, hd, ps = case["B"], case["R"], case["Hkv"], case["hd"], case["ps"]
    L = st["max_len"]
    t = torch.arange(L, device="cuda")
    page = st["table"].long()[:, t // ps].clamp(min=0)
    row = (t % ps).expand(B, L)
    if "k_scale" in st:
        K = _values(st["k"][page, :, row], st["k_scale"][page, :, row], st["k_global"])
        V = _values(st["v"][page, :, row], st["v_scale"][page, :, row], st["v_global"])
    else:
        K, V = st["k"][page, :, row].float(), st["v"][page, :, row].float()
    own_row = t[None, :] - st["lens"].long()[:, None]                      # [B, L]: which of the call's rows
    i = torch.arange(R, device="cuda")
    see = own_row[:, None, :] <= i[None, :, None]                          # causal
    if st["mask"] is not None:
        m = torch.gather(st["mask"].bool(), 2, own_row.clamp(0, R - 1)[:, None, :].expand(B, R, L))
        see = (own_row[:, None, :] < 0) | (m & (own_row[:, None, :] < R))
    q = st["q"].float().reshape(B, R, Hkv, -1, hd).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, hd)
    s = torch.matmul(q, K.permute(0, 2, 3, 1)).unflatten(2, (-1, R)) / math.sqrt(hd)
    s = s.masked_fill(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul((p / z).flatten(2, 3), V.transpose(1, 2)).unflatten(2, (-1, R))
    lse = (top + z.log())[..., 0]
    return (o.permute(0, 3, 1, 2, 4).reshape(B * R, -1, hd).to(torch.bfloat16).contiguous(),
            lse.permute(0, 3, 1, 2).reshape(B * R, -1).contiguous())


def run(st):
    case, op = st["case"], st["op"]
    if own:
        return _run_own(st)
    if op == "rotary":
        return _rotate(st["x"], st["positions"], st["inv_freq"], case["inter"]).to(st["x"].dtype)
    if op == "append":
        rot = [_rotate(st[n], st["positions"], st["inv_freq"], case["inter"]).to(torch.bfloat16) for n in ("q_rows", "k_rows")]
        page, row = _place(st, case["R"])
        if case["kind"] == "bf16":
            st["k"][page, :, row] = rot[1]
            st["v"][page, :, row] = st["v_rows"]
            return rot[0], st["k"], st["v"]
        st["k"][page, :, row], st["k_scale"][page, :, row] = _quantise(rot[1], st["k_global"])
        st["v"][page, :, row], st["v_scale"][page, :, row] = _quantise(st["v_rows"], st["v_global"])
        return (rot[0],) + _packed(st)
    if op == "gather":
        return _packed(st)
    if op == "attention":
        return _attend(st)
    # accept: slot s of request b's tree sits behind its cached keys at lens[b] + s; the
    # accepted slots move to lens[b] + 1, lens[b] + 2, ...
    ps, S, lens = case["ps"], case["S"], st["lens"].long()
    j = torch.arange(S, device="cuda")
    take = j[None, :] < st["accept_len"].long()[:, None]
    to = (lens[:, None] + 1 + j).clamp(max=case["ps"] * st["table"].shape[1] - 1)
    src = lens[:, None] + torch.where(take, st["accept_slots"].long(), 0)
    dst = torch.where(take, to, lens[:, None])                             # the rest: the root onto itself
    src = torch.where(take, src, lens[:, None])
    table = st["table"].long()
    sp, sr, dp, dr = torch.gather(table, 1, src // ps), src % ps, torch.gather(table, 1, dst // ps), dst % ps
    st["k"][:, dp, :, dr] = st["k"][:, sp, :, sr]
    st["v"][:, dp, :, dr] = st["v"][:, sp, :, sr]
    return st["k"], st["v"], (st["lens"] + 1 + st["accept_len"]).to(torch.int32)


def _run_own(st):
    from eagle_speculative_decoding_03_gb300 import binding as eb
    case, op = st["case"], st["op"]
    if op == "rotary":
        return eb.rotary(st["x"], st["positions"], st["rope"])
    if op == "append":
        q = eb.kv_append(st["cache"], st["k_rows"], st["v_rows"], st["cu_rows"], st["lens"], positions=st["positions"],
                         rope=st["rope"], q=st["q_rows"])
        if case["kind"] == "bf16":
            return q, st["k"], st["v"]
        return (q,) + eb.kv_gather(st["cache"], st["cu_seqlens"], st["total"])
    if op == "gather":
        return eb.kv_gather(st["cache"], st["cu_seqlens"], st["total"])
    if op == "attention":
        return eb.kv_attention(st["cache"], st["q"], st["cu_rows"], st["lens"], max_rows=case["R"], max_len=st["max_len"],
                               mask=st["mask"], lse=True)
    return st["k"], st["v"], eb.kv_accept(st["cache"], st["lens"], st["accept_len"], st["accept_slots"])


# ------------------------------------------------------------------- work and exact values
def work(case):
    op = case["op"]
    if op == "rotary":
        e = case["N"] * case["H"] * case["hd"]
        return {"bytes": 2 * e * (2 if case["dtype"] == "bf16" else 4) + 4 * case["N"],
                "flops": 3 * case["N"] * case["H"] * case["rot"]}
    B, Hkv, hd = case["B"], case["Hkv"], case["hd"]
    per = 2 * Hkv * (2 * hd if case.get("kind", "bf16") == "bf16" else hd // 2 + hd // 16)   # a token's key and value
    ctx = sum(_ctx(case))
    if op == "append":
        N = B * case["R"]
        b = N * (2 * hd * (2 * case["Hq"] + 2 * Hkv) + per + 4)
        if case["kind"] == "f4":
            b += (ctx + N) * (per + 4 * Hkv * hd)
        return {"bytes": b, "flops": 3 * N * (case["Hq"] + Hkv) * case["rot"]}
    if op == "gather":
        return {"bytes": ctx * (per + 4 * Hkv * hd), "flops": 0}
    if op == "attention":
        R, Hq = case["R"], case["Hq"]
        seen = R * ctx + B * (R * (R + 1) // 2)                            # (a tree's rows see no more)
        return {"bytes": (ctx + B * R) * per + B * R * Hq * (4 * hd + 4) + (B * R * R if case["tree"] else 0),
                "flops": 4 * hd * Hq * seen}
    moved = sum(_dst_span(case))
    return {"bytes": 2 * moved * per * case["L"] + B * (4 * case["S"] + 12), "flops": 0}


def exact(case, seed):
    """The operators from their definitions in 64 bits, request by request."""
    st = prepare(case, seed)
    op = case["op"]

    def turn(x, pos, rot, theta, inter):
        x = x.double().clone()
        half = rot // 2
        w = pos.double().view(-1, 1, 1) / theta ** (torch.arange(half, device="cuda").double() * 2 / rot)
        first = torch.arange(half, device="cuda") * (2 if inter else 1)
        second = first + (1 if inter else half)
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(w), w)
        x[..., first], x[..., second] = z.real, z.imag
        return x

    def four(x, glob):
        """The values that bf16 numbers become in 4 bits: nearest magnitude, even code on a tie."""
        x = x.double()
        out = torch.empty_like(x)
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device="cuda")      # even codes win ties
        for g0 in range(0, x.shape[-1], 16):
            y = x[..., g0:g0 + 16]
            sc = (y.abs().max(-1).values / (6 * glob)).clamp(max=448).float().to(torch.float8_e4m3fn).double()
            u = (sc * glob)[..., None]
            off = (y.abs()[..., None] - u[..., None] * grid[order]).abs()
            out[..., g0:g0 + 16] = grid[order][off.argmin(-1)] * u * torch.sign(y)
        return out

    if op == "rotary":
        return turn(st["x"], st["positions"], case["rot"], case["theta"], case["inter"])
    ps, Hkv, hd, ctx = case["ps"], case["Hkv"], case["hd"], _ctx(case)

    def held(b, n, name):
        """Request b's first n keys or values, [n, Hkv, hd]."""
        pages = st["table"][b, :(n + ps - 1) // ps].long()
        def rows(x):
            return x[pages].transpose(1, 2).flatten(0, 1)[:n]
        if name + "_scale" not in st:
            return rows(st[name]).double()
        c = rows(st[name]).int()
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        mag = torch.empty(c.shape[:-1] + (hd,), dtype=torch.float64, device="cuda")
        mag[..., 0::2] = grid[c & 7] * (1 - 2 * ((c >> 3) & 1))
        mag[..., 1::2] = grid[(c >> 4) & 7] * (1 - 2 * (c >> 7))
        sc = rows(st[name + "_scale"]).view(torch.float8_e4m3fn).double() * st[name + "_global"]
        return mag * sc.repeat_interleave(16, -1)

    if op == "append":
        R = case["R"]
        q = turn(st["q_rows"], st["positions"], case["rot"], case["theta"], case["inter"])
        k = turn(st["k_rows"], st["positions"], case["rot"], case["theta"], case["inter"])
        v = st["v_rows"].double()
        if case["kind"] == "f4":                                           # (an empty cache: its rows are the call's)
            return q, four(k.to(torch.bfloat16), st["k_global"]), four(v, st["v_global"])
        kp, vp = st["k"].double(), st["v"].double()
        for b, n in enumerate(ctx):
            for i in range(R):
                p, r = int(st["table"][b, (n + i) // ps]), (n + i) % ps
                kp[p, :, r], vp[p, :, r] = k[b * R + i], v[b * R + i]
        return q, kp, vp
    if op == "gather":
        return tuple(torch.cat([held(b, n, name) for b, n in enumerate(ctx)]) for name in ("k", "v"))
    if op == "attention":
        R, G = case["R"], case["Hq"] // Hkv
        if work(case)["flops"] > 4e11:
            return None
        out, lses = [], []
        for b, n in enumerate(ctx):
            K, V = held(b, n + R, "k"), held(b, n + R, "v")
            q = st["q"][b * R:(b + 1) * R].double()
            sees = torch.ones(R, n + R, dtype=torch.bool, device="cuda")
            sees[:, n:] = st["mask"][b].bool() if st["mask"] is not None else torch.ones(R, R, device="cuda").tril().bool()
            o, l = torch.empty_like(q), torch.empty(R, case["Hq"], dtype=torch.float64, device="cuda")
            for h in range(case["Hq"]):
                s = (q[:, h] @ K[:, h // G].T) * hd ** -0.5
                s[~sees] = -math.inf
                l[:, h] = torch.logsumexp(s, 1)
                o[:, h] = torch.exp(s - l[:, h:h + 1]) @ V[:, h // G]
            out.append(o)
            lses.append(l)
        return torch.cat(out), torch.cat(lses)
    k, v = st["k"].double(), st["v"].double()
    kept = st["accept_slots"].tolist()
    for b, n in enumerate(ctx):
        for j in range(int(st["accept_len"][b])):
            s, d = n + kept[b][j], n + 1 + j
            ps_, pd = int(st["table"][b, s // ps]), int(st["table"][b, d // ps])
            k[:, pd, :, d % ps], v[:, pd, :, d % ps] = k[:, ps_, :, s % ps], v[:, ps_, :, s % ps]
    return k, v, None
