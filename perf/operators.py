"""The 4-bit key/value cache operators: what is measured, and their plain forms.

Two operators on a paged cache that holds keys and values in 4 bits:

* "cache": new K and V rows are quantised as they are written into the pages of
  their sequences, and the same tokens are read back as bf16;
* "attention": queries (one per sequence in a decode step, a few when drafted
  tokens are checked, hundreds for a chunk of a prompt) against the cache.

Format of a value: along the head dimension, groups of ``group`` values share
a bf16 scale and a bf16 minimum and are held as codes 0..15,

    min = the group's least value,   scale = bf16((max / 2 - min / 2) * f32(2/15)),
    code = rint((x / 2 - min / 2) * (1 / (scale / 2)))   clamped to 0..15,
    value = min + scale * code,

the code decided in float32, each operation rounded once (scale below 2^-126:
0, and code 0; a group with a NaN or an infinity: scale and min NaN).

Layout: cache uint8 [pages, kv_heads, page_size / 16 * cell]; a cell holds 16
tokens of one head: K codes [16][d/2], V codes [16][d/2], K parameters
[16][d/group] (scale, min) bf16 pairs, V parameters likewise.  A K row stores
its 32-bit words (8 codes, lowest nibble first) w = 4 j + c at place c (d/32) +
j; a V row stores its 16-bit halves q 8 + g at place g (d/32) + q, and the
32-byte sector s of the V codes stands at place (s & ~3) | ((s + (s >> 2)) & 3).
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def listed():
    return [
        # one user, a short chat, a small model: nothing but latency
        dict(name="decode 1x200 d64", op="attention", B=1, Nq=1, lo=200, hi=200, H=16, kv=2, d=64,
             group=64, page=16, causal=True, packed=False),
        # a serving batch of ragged lengths, grouped heads: the ordinary decode step
        dict(name="decode 64x8k ragged", op="attention", B=64, Nq=1, lo=300, hi=16000, H=32, kv=8,
             d=128, group=64, page=64, causal=True, packed=False),
        # one very long context: the split over the cache
        dict(name="decode 1x130001", op="attention", B=1, Nq=1, lo=130001, hi=130001, H=32, kv=8,
             d=128, group=128, page=128, causal=True, packed=False),
        # as many heads of keys as of queries, small heads
        dict(name="decode mha 32x4k d64", op="attention", B=32, Nq=1, lo=1, hi=8191, H=16, kv=16,
             d=64, group=32, page=32, causal=True, packed=False),
        # many short chats, small pages, some slots of the batch idle (length 0)
        dict(name="decode 256x1k", op="attention", B=256, Nq=1, lo=0, hi=2047, H=32, kv=8, d=128,
             group=32, page=16, causal=True, packed=False),
        # drafted tokens checked: four queries a sequence, causal among themselves
        dict(name="verify 16x4 on 16k", op="attention", B=16, Nq=4, lo=1000, hi=20000, H=32, kv=4,
             d=128, group=64, page=64, causal=True, packed=False),
        # chunks of prompts on what is cached already, ragged and packed
        dict(name="chunk 4x512 on 16k", op="attention", B=4, Nq=512, lo=2049, hi=16384, H=32, kv=8,
             d=128, group=128, page=64, causal=True, packed=True),
        # one user's new token, then a serving batch's
        dict(name="write 1x1 d64", op="cache", B=1, Nq=1, lo=200, hi=200, H=16, kv=2, d=64,
             group=64, page=16, fused=False),
        dict(name="write 64x1", op="cache", B=64, Nq=1, lo=300, hi=16000, H=32, kv=8, d=128,
             group=64, page=64, fused=True),
        # prompts of ragged lengths, K and V still in the fused projection's rows
        dict(name="write 8 prompts", op="cache", B=8, Nq=4000, lo=4000, hi=4500, H=32, kv=8, d=128,
             group=32, page=16, fused=True),
        # long prompts at once, one scale a row: bandwidth and nothing else
        dict(name="write 32 prompts", op="cache", B=32, Nq=8191, lo=8192, hi=9000, H=16, kv=4,
             d=128, group=128, page=128, fused=False),
    ]


def draw(rng):
    d = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    size = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    B = size(1, 256)
    if rng.random() < 0.35:
        n = min(size(1, 8192), max(1, 130_000_000 // (B * kv * d)))
        lo = n + size(1, 4000) - 1
        return dict(op="cache", B=B, Nq=n, lo=lo, hi=lo + size(1, 1000), H=kv * rng.choice([1, 4]),
                    kv=kv, d=d, group=group, page=page, fused=rng.random() < 0.5)
    hi = min(size(1, 130_000), max(1, 1_000_000_000 // (B * kv * d)))
    H = kv * rng.choice([1, 2, 3, 4, 7, 8, 16])
    Nq = 1 if rng.random() < 0.5 else size(2, 512)
    Nq = max(1, min(Nq, 400_000_000 // (B * H * hi), hi))
    return dict(op="attention", B=B, Nq=Nq, lo=rng.choice([0, hi // 3, hi]), hi=hi, H=H, kv=kv, d=d,
                group=group, page=page, causal=rng.random() < 0.7, packed=rng.random() < 0.4)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], in no order, the same for every seed; both ends occur where n > 1."""
    v = [lo + int((hi - lo + 1) * ((0.6180339887 * i + 0.35) % 1.0)) for i in range(n)]
    v[0] = hi
    if n > 1:
        v[n // 2] = lo
    return v


def _sizes(case):
    """(tokens in the cache after the call, new tokens or queries) of each sequence."""
    L = _spread(case["B"], case["lo"], case["hi"])
    if case["op"] == "cache":
        ragged = case["Nq"] > 1 and case["fused"]
    else:
        ragged = case["packed"]
    n = _spread(case["B"], (case["Nq"] + 1) // 2, case["Nq"])[::-1] if ragged else [case["Nq"]] * case["B"]
    return L, n


# ---- the format, in torch ---------------------------------------------------------

def _cell_bytes(d, group):
    return 16 * d + 128 * (d // group)


def _orders(d, device):
    """Byte places of the logical code bytes [16, d/2] within a cell: (of K, of V)."""
    t = torch.arange(16, device=device)[:, None]
    b = torch.arange(d // 2, device=device)[None, :]
    w, n = b // 4, d // 32
    k = t * (d // 2) + ((w % 4) * n + w // 4) * 4 + b % 4
    h = b // 2
    p = t * (d // 2) + ((h % 8) * n + h // 8) * 2 + b % 2
    s = p // 32
    v = 16 * (d // 2) + ((s & ~3) | ((s + (s >> 2)) & 3)) * 32 + p % 32
    return k, v


def _quantise(x, group):
    """Codes uint8 [..., d] and (scale, min) bf16 [..., d/group, 2]."""
    g = x.float().unflatten(-1, (-1, group))
    hi, lo = g.amax(-1, keepdim=True), g.amin(-1, keepdim=True)
    scale = ((hi * 0.5 - lo * 0.5) * (2.0 / 15.0)).to(BF16)
    scale = torch.where(scale.float() < 2.0 ** -126, torch.zeros_like(scale), scale)
    bad = ~(torch.isfinite(hi) & torch.isfinite(lo))
    r = torch.where(scale > 0, 1.0 / (scale.float() * 0.5), torch.zeros_like(hi))
    code = torch.round((g * 0.5 - lo * 0.5) * r).clamp(0, 15).nan_to_num(0)
    pair = torch.cat((scale.float(), lo), -1).masked_fill(bad, math.nan).to(BF16)
    return code.to(torch.uint8).flatten(-2), pair


def _value(code, pair, group):
    """float32 values of codes [..., d] with pairs [..., d/group, 2]."""
    g = code.float().unflatten(-1, (-1, group))
    return (pair[..., 1:].float() + pair[..., :1].float() * g).flatten(-2)


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _rows(state, n, total):
    """Sequence and place within it of each of `total` packed rows, the last n[b] tokens of sequence b."""
    cu, L = state["cu"].long(), state["seqlens"].long()
    r = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu, r, right=True) - 1
    return b, L[b] - (cu[b + 1] - cu[b]) + (r - cu[b])


def _places(state, d, group, page, kv):
    """Byte index in the flat cache of each new row's K codes, V codes, K pairs, V pairs."""
    b, pos = _rows(state, state["n"], state["total"])
    cell = _cell_bytes(d, group)
    pg = state["table"][b, pos // page].long()
    h = torch.arange(kv, device=pg.device)
    base = ((pg[:, None] * kv + h) * (page // 16) + (pos % page // 16)[:, None]) * cell
    ko, vo = _orders(d, pg.device)
    t = pos % 16
    par = 16 * d + t[:, None] * (d // group) * 4 + torch.arange(d // group * 4, device=pg.device)
    return (base[..., None] + ko[t][:, None], base[..., None] + vo[t][:, None],
            base[..., None] + par[:, None], base[..., None] + par[:, None] + 64 * (d // group))


def _plain_cache(state):
    c = state["case"]
    d, group = c["d"], c["group"]
    flat = state["cache"].view(-1)
    ik, iv, ipk, ipv = _places(state, d, group, c["page"], c["kv"])
    for x, i, ip in ((state["k"], ik, ipk), (state["v"], iv, ipv)):
        code, pair = _quantise(x, group)
        flat[i] = code[..., 0::2] | (code[..., 1::2] << 4)
        flat[ip] = pair.contiguous().view(torch.uint8).flatten(-2)
    out = []
    for i, ip in ((ik, ipk), (iv, ipv)):
        pair = flat[ip].view(BF16).unflatten(-1, (-1, 2))
        out.append(_value(_nibbles(flat[i]), pair, group).to(BF16))
    return {"k": out[0], "v": out[1]}


def _plain_attention(state):
    c = state["case"]
    d, group, kv, H, B = c["d"], c["group"], c["kv"], c["H"], c["B"]
    L, cu = state["seqlens"].long(), state["cu"].long()
    # the cells of every sequence's pages, decoded: [B, tokens, kv, d]
    cells = state["cache"][state["table"].long().clamp(min=0)].unflatten(-1, (-1, _cell_bytes(d, group)))
    kv32 = []
    for k, o in enumerate(_orders(d, L.device)):
        at = 16 * d + 64 * (d // group) * k
        pair = cells[..., at:at + 64 * (d // group)].contiguous().view(BF16).unflatten(-1, (16, d // group, 2))
        x = _value(_nibbles(cells[..., o]), pair, group)           # [B, pages, kv, cells, 16, d]
        kv32.append(x.permute(0, 2, 1, 3, 4, 5).reshape(B, kv, -1, d))
    K, V = kv32
    T = K.shape[2]
    # queries, padded to one count: [B, kv, H / kv * Nq, d]
    nq = cu[1:] - cu[:-1]
    i = torch.arange(c["Nq"], device=L.device)
    row = (cu[:-1, None] + torch.minimum(i, nq[:, None] - 1)).clamp(min=0)
    q = state["q"].reshape(-1, H, d)[row].float().reshape(B, -1, kv, H // kv, d).permute(0, 2, 3, 1, 4)
    s = (q.reshape(B, kv, -1, d) @ K.transpose(-1, -2) / math.sqrt(d)).unflatten(2, (H // kv, -1))
    j = torch.arange(T, device=L.device)
    seen = j < (L[:, None, None] - nq[:, None, None] + i[:, None] + 1 if c["causal"] else L[:, None, None])
    seen = (seen & (j < L[:, None, None]))[:, None, None]
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True).nan_to_num(0, 0, 0) if T else s.new_zeros(*s.shape[:-1], 1)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ V).unflatten(2, (H // kv, -1)) / torch.where(z > 0, z, 1)
    lse = (m + torch.log(z))[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, -1, H, d).to(BF16), lse.permute(0, 3, 1, 2).reshape(B, -1, H)
    if c["packed"]:
        b, at = _rows(state, state["n"], state["total"])
        at = at - (L - nq)[b]
        return {"o": o[b, at], "lse": lse[b, at].transpose(0, 1).contiguous()}
    return {"o": o, "lse": lse.transpose(1, 2).contiguous()}


# ---- inputs ------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev, dtype=F32)  # noqa: E731
    d, group, page, kv, H, B = (case[k] for k in ("d", "group", "page", "kv", "H", "B"))
    L, n = _sizes(case)
    cell = _cell_bytes(d, group)
    per = [(x + page - 1) // page for x in L]
    pages, width = sum(per) + 1, max(1, max(per))
    # the pages of the sequences lie in the pool in no order; places of the table behind a sequence's end hold -1
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    first = torch.tensor([0] + per, device=dev).cumsum(0)
    col = torch.arange(width, device=dev)
    used = col < torch.tensor(per, device=dev)[:, None]
    table = torch.where(used, order[(first[:-1, None] + col).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    cu = torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32)
    state = dict(case=dict(case), seqlens=torch.tensor(L, device=dev, dtype=torch.int32), table=table, cu=cu,
                 n=max(n), total=sum(n), longest=max(L))
    # keys have channels with an offset of their own, as after a biased projection
    off = normal(2, kv, 1, d) * torch.tensor([1.5, 0.1], device=dev)[:, None, None, None]
    cache = torch.empty((pages, kv, page // 16 * cell), dtype=torch.uint8, device=dev)
    if case["op"] == "attention":
        ko, vo = _orders(d, dev)
        step = max(1, 40_000_000 // (kv * page * d))
        for p in range(0, pages, step):
            part = cache[p:p + step].unflatten(-1, (-1, cell))
            for k, o in enumerate((ko, vo)):
                x = (normal(len(part), kv, page, d) + off[k]).to(BF16)
                code, pair = _quantise(x, group)
                code = (code[..., 0::2] | (code[..., 1::2] << 4)).unflatten(2, (-1, 16)).flatten(-2)
                part[..., o.flatten()] = code
                at = 16 * d + 64 * (d // group) * k
                part[..., at:at + 64 * (d // group)] = pair.contiguous().view(torch.uint8).reshape(*part.shape[:3], -1)
        q = (normal(sum(n), H, d) * 1.5).to(BF16)
        state["q"] = q if case["packed"] else q.view(B, case["Nq"], H, d)
    else:
        cache.zero_()
        T = sum(n)
        kk, vv = ((normal(T, kv, d) + off[i, :, 0]).to(BF16) for i in (0, 1))
        if case["fused"]:
            rows = normal(T, H + 2 * kv, d).to(BF16)
            rows[:, H:H + kv], rows[:, H + kv:] = kk, vv
            kk, vv = rows[:, H:H + kv], rows[:, H + kv:]
        state["k"], state["v"] = kk, vv
    state["cache"] = cache
    return state


def run(state):
    c = state["case"]
    if not own:
        return _plain_cache(state) if c["op"] == "cache" else _plain_attention(state)
    import online_softmax_06_gb300 as fa
    if c["op"] == "cache":
        where = dict(cu_seqlens=state["cu"], max_new=state["n"], group=c["group"])
        fa.kv4_append(state["k"], state["v"], state["cache"], state["table"], state["seqlens"], **where)
        k, v = fa.kv4_read(state["cache"], state["table"], state["seqlens"], total=state["total"], d=c["d"], **where)
        return {"k": k, "v": v}
    packed = dict(cu_seqlens=state["cu"], max_q=state["n"]) if c["packed"] else {}
    o, lse = fa.attention_kv4(state["q"], state["cache"], state["table"], state["seqlens"], max_seqlen=state["longest"],
                              group=c["group"], causal=c["causal"], **packed)
    return {"o": o, "lse": lse}


def work(case):
    L, n = _sizes(case)
    d, kv, H = case["d"], case["kv"], case["H"]
    row = kv * _cell_bytes(d, case["group"]) // 16                # cache bytes of a token
    if case["op"] == "cache":
        T = sum(n)
        return {"bytes": T * (2 * 4 * kv * d + 2 * row), "flops": 12 * T * kv * d}
    seen = 0
    for x, q in zip(L, n):
        if case["causal"]:                                        # query i of q sees x - q + 1 + i keys, none below 0
            a = max(0, q - x)
            seen += (q - a) * (x - q + 1 + a + x) // 2
        else:
            seen += q * x
    T = sum(n)
    return {"bytes": sum(L) * row + T * H * (4 * d + 4) + 4 * sum((x + case["page"] - 1) // case["page"] for x in L),
            "flops": 4 * d * H * seen}


def exact(case, seed):
    s = prepare(case, seed)
    d, group, page, kv, H = (case[k] for k in ("d", "group", "page", "kv", "H"))
    if case["op"] == "cache":
        out = {}
        for name in ("k", "v"):
            parts = []
            for x in s[name].split(8192):                         # float32 steps of the definition, each rounded once from 64 bits
                g = x.to(F64).reshape(x.shape[0], kv, d // group, group)
                lo = g.min(3, keepdim=True).values
                half = ((g.max(3, keepdim=True).values - lo) / 2).to(F32).to(F64)
                c15 = float(torch.tensor(2 / 15, dtype=F32))
                sc = (half * c15).to(F32).to(BF16).to(F64)
                sc[sc < 2.0 ** -126] = 0
                inv = (2 / sc).to(F32).to(F64)
                inv[sc == 0] = 0
                u = (((g - lo) / 2).to(F32).to(F64) * inv).to(F32).to(F64).round().clamp(0, 15)
                parts.append((lo + sc * u).reshape(x.shape))
            out[name] = torch.cat(parts)
        return out
    # where value i of token t stands in a cell: byte, and whether in its upper half
    cell, n = _cell_bytes(d, group), d // 32
    dev = s["cache"].device
    byte, up = torch.zeros(2, 16, d, dtype=torch.long), torch.arange(d) % 2 == 1
    for t in range(16):
        for i in range(d):
            w = i // 8                                            # K: 32-bit words
            byte[0, t, i] = t * (d // 2) + ((w % 4) * n + w // 4) * 4 + (i % 8) // 2
            h = i // 4                                            # V: 16-bit halves, rotated 32-byte sectors
            a = t * (d // 2) + ((h % 8) * n + h // 8) * 2 + (i % 4) // 2
            line, sector = a // 128, a % 128 // 32
            byte[1, t, i] = 8 * d + line * 128 + (sector + line) % 4 * 32 + a % 32
    byte, up = byte.to(dev), up.to(dev)
    L, nq = _sizes(case)
    q = s["q"].reshape(-1, H, d)
    o = torch.zeros(q.shape, dtype=F64, device=dev)
    lse = torch.full((q.shape[0], H), -math.inf, dtype=F64, device=dev)
    at = 0
    for b, (x, m) in enumerate(zip(L, nq)):
        rows, at = slice(at, at + m), at + m
        if x == 0:
            continue
        pg = s["cache"][s["table"][b, :(x + page - 1) // page].long()].reshape(-1, kv, page // 16, cell)
        for h in range(kv):
            c = pg[:, h].reshape(-1, cell)                        # the cells in the order of the tokens
            x32 = []
            for k in (0, 1):
                raw = c[:, byte[k]].long()
                code = torch.where(up, raw // 16, raw % 16)
                a = 16 * d + 64 * (d // group) * k
                par = c[:, a:a + 64 * (d // group)].contiguous().view(BF16).reshape(-1, 16, d // group, 2).to(F64)
                par = par.repeat_interleave(group, 2)
                x32.append((par[..., 0] * code + par[..., 1]).reshape(-1, d)[:x])
            hs = slice(h * (H // kv), (h + 1) * (H // kv))
            for r0 in range(0, m, 64):
                r1 = min(m, r0 + 64)
                qq = q[rows][r0:r1, hs].to(F64)
                sc = torch.einsum("ihd,jd->ihj", qq, x32[0]) / math.sqrt(d)
                if case["causal"]:
                    last = torch.arange(r0, r1, device=dev) + (x - m)
                    sc = sc.masked_fill((torch.arange(x, device=dev) > last[:, None])[:, None], -math.inf)
                z = torch.logsumexp(sc, -1)
                p = torch.exp(sc - torch.where(torch.isfinite(z), z, 0.0)[..., None])
                o[rows][r0:r1, hs] = torch.einsum("ihj,jd->ihd", p, x32[1])
                lse[rows][r0:r1, hs] = z
    if case["packed"]:
        return {"o": o, "lse": lse.t().contiguous()}
    B = case["B"]
    return {"o": o.view(B, -1, H, d), "lse": lse.view(B, -1, H).transpose(1, 2).contiguous()}
