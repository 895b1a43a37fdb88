"""Window attention and the norm and rotation before it: what is measured, and their plain forms.

Two operators of an attention layer:

* "window": attention with a sliding window and a few first tokens that stay
  visible (sinks).  Query i of the n last tokens of a sequence of L keys sits at
  p = i + L - n and sees key j iff j <= p and (j > p - window or j < sinks).
  Query head h reads kv head h / (H / kv).  With grad, a training step: the
  gradients of sum(dO * O) with respect to Q, K and V as well.  A row that sees
  no key has O = 0 and lse = -inf.
* "rope": each head of Q and K normed, x / sqrt(mean(x^2) + eps) * weight, and
  its first `rot` values rotated by pos * inv_freq[j], in pairs (j, j + rot / 2)
  or (2 j, 2 j + 1).  With grad the gradients with respect to Q, K and both
  weights.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def listed():
    return [
        # one user, a short chat, a small model: nothing but latency
        dict(name="window decode 1x600 d64", op="window", form="cache", B=1, Nq=1, lo=600, hi=600, H=16, kv=2, d=64,
             window=256, sinks=4, grad=False),
        # a serving batch of ragged lengths over a bf16 cache, grouped heads: the ordinary decode step
        dict(name="window decode 64x16k", op="window", form="cache", B=64, Nq=1, lo=300, hi=16000, H=32, kv=8, d=128,
             window=4096, sinks=4, grad=False),
        # one long context and many kv heads: the window split over the GPU
        dict(name="window decode 1x32k", op="window", form="cache", B=1, Nq=1, lo=32001, hi=32001, H=32, kv=8, d=128,
             window=8192, sinks=4, grad=False),
        # drafted tokens checked: four queries a sequence
        dict(name="window verify 16x4", op="window", form="cache", B=16, Nq=4, lo=500, hi=9000, H=32, kv=4, d=128,
             window=1024, sinks=16, grad=False),
        # chunks of prompts on what is there already, ragged and packed
        dict(name="window chunk 4x512", op="window", form="packed", B=4, Nq=512, lo=2049, hi=16384, H=32, kv=8, d=128,
             window=4096, sinks=4, grad=False),
        # a training step of the benchmark's shape, grouped heads
        dict(name="window train 2x4096", op="window", form="dense", B=2, Nq=4096, lo=4096, hi=4096, H=32, kv=8, d=128,
             window=1024, sinks=4, grad=True),
        # long documents: the sinks are seen by every query
        dict(name="window train 1x32k", op="window", form="dense", B=1, Nq=32768, lo=32768, hi=32768, H=16, kv=4,
             d=128, window=2048, sinks=4, grad=True),
        # ragged packed sequences, as many kv heads as query heads, a narrow window and no sinks
        dict(name="window train packed d64", op="window", form="packed", B=8, Nq=3001, lo=0, hi=0, H=16, kv=16, d=64,
             window=256, sinks=0, grad=True),
        # one user's new token
        dict(name="rope 1 token d64", op="rope", T=1, H=16, kv=2, d=64, rot=64, interleaved=False, far=600,
             fused=True, grad=False),
        # a serving batch's new tokens at far positions
        dict(name="rope 64 tokens", op="rope", T=64, H=32, kv=8, d=128, rot=128, interleaved=False, far=1000000,
             fused=True, grad=False),
        # a training step of 32768 tokens: bandwidth and nothing else
        dict(name="rope train 32768", op="rope", T=32768, H=32, kv=8, d=128, rot=128, interleaved=False, far=4096,
             fused=True, grad=True),
        # half of each head rotated, in neighbouring pairs, an odd count of tokens and heads
        dict(name="rope train 5005 d64", op="rope", T=5005, H=15, kv=5, d=64, rot=32, interleaved=True, far=131072,
             fused=False, grad=True),
    ]


# what a drawn case may cost: the largest listed ones, in query-key pairs of heads, in values of Q (window) and of Q and K
_PAIRS, _ROWS, _VALUES = 1_000_000_000, 67_000_000, 160_000_000


def draw(rng):
    d = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    size = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    if rng.random() < 0.4:
        H = kv * rng.choice([1, 2, 3, 4, 7, 8])
        T = size(1, max(1, _VALUES // ((H + kv) * d)))
        return dict(op="rope", T=T, H=H, kv=kv, d=d, rot=rng.choice([d, d, d // 2, d // 4, 0]),
                    interleaved=rng.random() < 0.4, far=size(1, 4_000_000), fused=rng.random() < 0.5,
                    grad=rng.random() < 0.5)
    H = kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    window, sinks = size(1, 8192), rng.choice([0, 0, 1, 4, 4, 16, 64, 130, 300])
    kind = rng.choice(["decode", "decode", "verify", "chunk", "train", "train"])
    if kind in ("decode", "verify"):
        B = size(1, 128)
        hi = min(size(1, 40000), max(1, 400_000_000 // (B * kv * d)))
        return dict(op="window", form="cache", B=B, Nq=1 if kind == "decode" else rng.randint(2, 8),
                    lo=rng.choice([0, hi // 3, hi]), hi=hi, H=H, kv=kv, d=d, window=window, sinks=sinks, grad=False)
    B = size(1, 16)
    most = min(16384, max(1, _PAIRS // (B * H * (window + sinks))), max(1, _ROWS // (B * H * d)))
    if kind == "chunk":
        Nq = size(1, max(1, min(2048, most)))
        hi = Nq + size(1, 16000)
        return dict(op="window", form="packed", B=B, Nq=Nq, lo=rng.choice([hi // 2, hi]), hi=hi, H=H, kv=kv, d=d,
                    window=window, sinks=sinks, grad=False)
    # (a query that sees a single key has the gradient zero, and its computed one nothing but rounding: not alone)
    return dict(op="window", form=rng.choice(["dense", "packed"]), B=B, Nq=size(4, max(4, most)), lo=0, hi=0, H=H,
                kv=kv, d=d, window=max(8, window), sinks=sinks, grad=True)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], in no order, the same for every seed; both ends occur where n > 1."""
    v = [lo + int((hi - lo + 1) * ((0.6180339887 * i + 0.35) % 1.0)) for i in range(n)]
    v[0] = hi
    if n > 1:
        v[n // 2] = lo
    return v


def _sizes(case):
    """(keys, queries) of each sequence of a window case; with grad they are the same tokens."""
    B, n = case["B"], [case["Nq"]] * case["B"]
    if case["form"] == "packed":
        n = _spread(B, (case["Nq"] + 1) // 3, case["Nq"])[::-1]
    if case["grad"] or case["form"] == "dense":
        return n, n
    return _spread(B, case["lo"], case["hi"]), n


# ---- plain forms -------------------------------------------------------------------

def _heads(x, G):
    """[keys, kv, d] -> [kv * G, keys, d] in float32."""
    return x.float().transpose(0, 1).repeat_interleave(G, 0)


def _blocks(state):
    """(sequence, its rows of Q, its rows of K, rows r0:r1 of the sequence, key positions): blocks of queries."""
    c = state["case"]
    q0 = k0 = 0
    for x, n, room in zip(state["L"], state["n"], state["room"]):
        for r0 in range(0, n, 512):
            r1 = min(n, r0 + 512)
            hi = max(0, r1 + x - n)                       # keys the block's last query reaches
            lo = min(hi, max(0, r0 + x - n - c["window"] + 1))
            s = min(c["sinks"], lo)
            dev = state["q"].device
            yield q0, k0, r0, r1, torch.cat((torch.arange(s, device=dev), torch.arange(lo, hi, device=dev))), x - n
        q0, k0 = q0 + n, k0 + room


def _scores(state, q, K, r0, r1, j, off):
    c = state["case"]
    s = q @ K.transpose(-1, -2) / math.sqrt(c["d"])
    p = torch.arange(r0, r1, device=j.device)[:, None] + off
    return torch.where((j <= p) & ((j > p - c["window"]) | (j < c["sinks"])), s, -math.inf)


def _plain_cache(state):
    """One or a few queries a sequence: the seen rows of the cache gathered, all sequences at once."""
    c = state["case"]
    kv, G, W, S, n = c["kv"], c["H"] // c["kv"], c["window"], c["sinks"], c["Nq"]
    K, V, q = state["k"], state["v"], state["q"]
    L = state["seqlens"].long()
    width = min(K.shape[1], W + n - 1)
    lo = (L - n - W + 1).clamp(min=0)[:, None]
    a = torch.arange(min(S, K.shape[1]), device=L.device)
    j = torch.cat((torch.where(a < lo, a, K.shape[1]), lo + torch.arange(width, device=L.device)), 1)   # [B, keys]
    at = j.clamp(max=K.shape[1] - 1)[..., None, None].expand(-1, -1, kv, c["d"])
    Ks, Vs = (torch.gather(x, 1, at).float().transpose(1, 2) for x in (K, V))                # [B, kv, keys, d]
    qq = q.float().unflatten(2, (kv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)               # [B, kv, G n, d]
    s = (qq @ Ks.transpose(-1, -2) / math.sqrt(c["d"])).unflatten(2, (G, n))
    p = torch.arange(n, device=L.device) + (L - n)[:, None]
    j, p = j[:, None], p[..., None]
    seen = (j <= p) & ((j > p - W) | (j < S))
    s = torch.where(seen[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    Vs = torch.where(seen.any(1)[:, None, :, None], Vs, 0.0)
    o = (e.flatten(2, 3) @ Vs).unflatten(2, (G, n)) / torch.where(z > 0, z, 1.0)
    lse = (m + torch.log(z))[..., 0]
    return {"o": o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(BF16), "lse": lse.flatten(1, 2).contiguous()}


def _plain_window(state):
    c = state["case"]
    H, kv, d = c["H"], c["kv"], c["d"]
    G = H // kv
    q, k, v = (state[x].reshape(-1, h, d) for x, h in (("q", H), ("k", kv), ("v", kv)))
    o = torch.empty((q.shape[0], H, d), dtype=F32, device=q.device)
    lse = torch.empty((H, q.shape[0]), dtype=F32, device=q.device)
    dq = dk = dv = None
    if c["grad"]:
        do = state["do"].reshape(-1, H, d)
        dq, dk, dv = torch.empty_like(o), torch.zeros(k.shape, device=q.device), torch.zeros(k.shape, device=q.device)
    for q0, k0, r0, r1, j, off in _blocks(state):
        rows, keys = slice(q0 + r0, q0 + r1), k0 + j
        qq, K, V = _heads(q[rows], 1), _heads(k[keys], G), _heads(v[keys], G)
        s = _scores(state, qq, K, r0, r1, j, off)
        m = s.amax(-1, keepdim=True) if len(j) else s.new_zeros(*s.shape[:-1], 1)
        m = torch.where(m == -math.inf, 0.0, m)
        e = torch.exp(s - m)
        z = e.sum(-1, keepdim=True)
        p = e / torch.where(z > 0, z, 1.0)
        oo = p @ V
        o[rows], lse[:, rows] = oo.transpose(0, 1), (m + torch.log(z))[..., 0]
        if c["grad"]:
            g = _heads(do[rows], 1)
            ds = p * (g @ V.transpose(-1, -2) - (g * oo).sum(-1, keepdim=True)) / math.sqrt(d)
            dq[rows] = (ds @ K).transpose(0, 1)
            for acc, x in ((dk, ds.transpose(-1, -2) @ qq), (dv, p.transpose(-1, -2) @ g)):
                acc[keys] += x.unflatten(0, (kv, G)).sum(1).transpose(0, 1)
    out = {"o": o.to(BF16).view(state["q"].shape)}
    out["lse"] = lse if c["form"] == "packed" else lse.view(H, c["B"], -1).transpose(0, 1).contiguous()
    if c["grad"]:
        out.update(dq=dq.to(BF16).view(state["q"].shape), dk=dk.to(BF16).view(state["k"].shape),
                   dv=dv.to(BF16).view(state["v"].shape))
    return out


def _rotate(x, cos, sin, rot, interleaved):
    """The first `rot` values of x [T, heads, d] turned by the angles of cos, sin [T, 1, rot / 2]."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_rope(state):
    c = state["case"]
    rot, pairs = c["rot"], c["interleaved"]
    ang = state["pos"].to(F64)[:, None, None] * state["freq"]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    out = {}
    for n in ("q", "k"):
        x, w = state[n].float(), state["w" + n]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        hat = x * r
        out[n] = _rotate(hat * w, cos, sin, rot, pairs).to(BF16)
        if c["grad"]:
            g = _rotate(state["d" + n].float(), cos, -sin, rot, pairs)
            out["dw" + n] = (g * hat).sum((0, 1), dtype=F64).float()
            g = g * w
            out["d" + n] = ((g - hat * (g * hat).mean(-1, keepdim=True)) * r).to(BF16)
    return out


# ---- inputs ------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev, dtype=F32)  # noqa: E731
    H, kv, d = case["H"], case["kv"], case["d"]
    state = dict(case=dict(case))
    if case["op"] == "rope":
        T, rot = case["T"], case["rot"]
        # a projection's rows: heads of unlike sizes, a few channels far larger than the others
        chan = torch.exp(normal(H + 2 * kv, d) * 0.5)
        if case["fused"]:
            rows = (normal(T, H + 2 * kv, d) * chan).to(BF16)
            state["q"], state["k"] = rows[:, :H], rows[:, H:H + kv]
        else:
            state["q"], state["k"] = ((normal(T, n, d) * chan[:n]).to(BF16) for n in (H, kv))
        state["wq"], state["wk"] = 1 + 0.3 * normal(d), 1 + 0.3 * normal(d)
        state["freq"] = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=F64) / max(rot, 1))
        # runs of neighbouring positions, as tokens of sequences are
        start = torch.randint(0, case["far"], (T // 512 + 1,), generator=gen, device=dev)
        state["pos"] = ((start[:, None] + torch.arange(512, device=dev)).flatten()[:T] % case["far"]).to(torch.int32)
        if case["grad"]:
            state["dq"], state["dk"] = (normal(T, n, d).to(BF16) for n in (H, kv))
        return state
    L, n = _sizes(case)
    B = case["B"]
    state.update(L=L, n=n, room=[case["hi"]] * B if case["form"] == "cache" else L, longest=max(L), most=max(n))
    # keys have channels with an offset of their own, as after a biased projection
    off = normal(2, kv, d) * torch.tensor([1.0, 0.1], device=dev)[:, None, None]
    T, Tk = sum(n), sum(state["room"])
    q, k, v = normal(T, H, d).to(BF16), torch.empty(Tk, kv, d, dtype=BF16, device=dev), torch.empty(
        Tk, kv, d, dtype=BF16, device=dev)
    for x, o in ((k, off[0]), (v, off[1])):
        for part in x.split(65536):
            part.copy_(normal(*part.shape) + o)
    if case["form"] == "packed":
        state["cu_q"], state["cu_k"] = (torch.tensor([0] + x, device=dev).cumsum(0).to(torch.int32) for x in (n, L))
    else:
        q, k, v = q.view(B, -1, H, d), k.view(B, -1, kv, d), v.view(B, -1, kv, d)
    if case["form"] == "cache":
        state["seqlens"] = torch.tensor(L, device=dev, dtype=torch.int32)
    if case["grad"]:
        state["do"] = normal(*q.shape).to(BF16)
    state.update(q=q, k=k, v=v)
    return state


def run(state):
    c = state["case"]
    if not own:
        return _plain_rope(state) if c["op"] == "rope" else (
            _plain_cache(state) if c["form"] == "cache" else _plain_window(state))
    import online_softmax_06_gb300 as fa
    if c["op"] == "rope":
        how = dict(positions=state["pos"], eps=EPS, interleaved=c["interleaved"])
        q, k = fa.qk_norm_rope_fwd(state["q"], state["k"], state["wq"], state["wk"], state["freq"], **how)
        if not c["grad"]:
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(state["q"], state["k"], state["dq"], state["dk"], state["wq"],
                                               state["wk"], state["freq"], **how)
        return {"q": q, "dwq": dwq, "dq": dq, "k": k, "dwk": dwk, "dk": dk}
    q, k, v = state["q"], state["k"], state["v"]
    how = dict(window=c["window"], sinks=c["sinks"])
    if c["grad"]:
        if c["form"] == "packed":
            how.update(cu_seqlens=state["cu_q"], max_seqlen=state["most"])
            fwd = dict(window=c["window"], sinks=c["sinks"], cu_seqlens_q=state["cu_q"], cu_seqlens_k=state["cu_q"],
                       max_q=state["most"], max_k=state["most"])
        else:
            fwd = how
        o, lse = fa.attention_window_fwd(q, k, v, **fwd)
        dq, dk, dv = fa.attention_window_bwd(q, k, v, o, state["do"], lse, **how)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if c["form"] == "cache":
        how.update(seqlens_k=state["seqlens"])
    else:
        how.update(cu_seqlens_q=state["cu_q"], cu_seqlens_k=state["cu_k"], max_q=state["most"], max_k=state["longest"])
    o, lse = fa.attention_window_fwd(q, k, v, **how)
    return {"o": o, "lse": lse}


def _seen(x, n, W, S):
    """(query-key pairs, keys seen by any) of n queries at the end of x keys."""
    i = torch.arange(max(0, n - x), n, dtype=torch.int64) + (x - n)       # positions that see something
    lo = (i - W + 1).clamp(min=0)
    pairs = int((i - lo + 1 + lo.clamp(max=S)).sum())
    if len(i) == 0:
        return 0, 0
    first = int(lo[0])
    return pairs, x - first + min(first, S)


def work(case):
    H, kv, d = case["H"], case["kv"], case["d"]
    if case["op"] == "rope":
        values = case["T"] * (H + kv) * d
        return {"bytes": values * (10 if case["grad"] else 4), "flops": values * (22 if case["grad"] else 8)}
    L, n = _sizes(case)
    pairs = keys = 0
    for x, m in zip(L, n):
        p, u = _seen(x, m, case["window"], case["sinks"])
        pairs, keys = pairs + p, keys + u
    T = sum(n)
    rows, cached = T * H * d * 2, keys * kv * d * 4                       # bytes of Q; of the seen K and V
    if not case["grad"]:
        return {"bytes": 2 * rows + cached + 4 * T * H, "flops": 4 * d * H * pairs}
    # Q, K, V, dO read, O and lse, dQ, dK, dV written
    return {"bytes": 4 * rows + 2 * cached + 4 * T * H, "flops": 14 * d * H * pairs}


# ---- the definitions in 64 bits -----------------------------------------------------

def _exact_rope(case, s):
    d, rot = case["d"], case["rot"]
    turn = torch.polar(torch.ones((), dtype=F64, device=s["pos"].device),
                       torch.outer(s["pos"].to(F64), s["freq"]))[:, None]           # complex [T, 1, rot / 2]
    out = {}
    for n in ("q", "k"):
        w = s["w" + n].to(F64).requires_grad_(case["grad"])
        ys, dxs, dw = [], [], torch.zeros(d, dtype=F64, device=w.device)
        for t in range(0, case["T"], 4096):
            part = slice(t, t + 4096)
            x = s[n][part].to(F64).requires_grad_(case["grad"])
            u = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w
            y = u
            if rot:
                z = u[..., :rot]
                z = z.unflatten(-1, (-1, 2)) if case["interleaved"] else z.unflatten(-1, (2, -1)).transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[part])
                z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
                y = torch.cat((z, u[..., rot:]), -1)
            ys.append(y.detach())
            if case["grad"]:
                gx, gw = torch.autograd.grad(y, (x, w), s["d" + n][part].to(F64))
                dxs.append(gx)
                dw += gw
        out[n] = torch.cat(ys)
        if case["grad"]:
            out["dw" + n], out["d" + n] = dw, torch.cat(dxs)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    H, kv, d, W, S, grad = (case[x] for x in ("H", "kv", "d", "window", "sinks", "grad"))
    L, n = _sizes(case)
    if sum(_seen(x, m, W, S)[0] for x, m in zip(L, n)) * H * d > 1e12:
        return None
    dev = s["q"].device
    q = s["q"].reshape(-1, H, d)
    k, v = (s[x].reshape(-1, kv, d) for x in ("k", "v"))
    o = torch.zeros(q.shape, dtype=F64, device=dev)
    lse = torch.full((H, len(q)), -math.inf, dtype=F64, device=dev)
    g = {}
    if grad:
        g = {x: torch.zeros(s[x].reshape(-1, h, d).shape, dtype=F64, device=dev) for x, h in (("q", H), ("k", kv), ("v", kv))}
    qa = ka = 0
    for x, m, room in zip(L, n, s["room"]):
        step = 1024 if W > 512 else 256
        for a in range(max(0, m - x), m, step):
            b = min(m, a + step)
            pos = torch.arange(a, b, device=dev) + (x - m)
            key = torch.arange(x, device=dev)
            key = key[(key <= pos[-1]) & ((key > pos[0] - W) | (key < S))]
            hidden = ~((key[None] <= pos[:, None]) & ((key[None] + W > pos[:, None]) | (key[None] < S)))
            for h in range(kv):
                hs = slice(h * (H // kv), (h + 1) * (H // kv))
                qq = q[qa + a:qa + b, hs].to(F64).requires_grad_(grad)
                kk, vv = (y[ka + key, h].to(F64).requires_grad_(grad) for y in (k, v))
                sc = torch.einsum("ihd,jd->hij", qq, kk).mul(d ** -0.5).masked_fill(hidden, -math.inf)
                oo = torch.einsum("hij,jd->ihd", torch.softmax(sc, -1), vv)
                o[qa + a:qa + b, hs], lse[hs, qa + a:qa + b] = oo.detach(), torch.logsumexp(sc, -1).detach()
                if grad:
                    up = s["do"].reshape(-1, H, d)[qa + a:qa + b, hs].to(F64)
                    gq, gk, gv = torch.autograd.grad(oo, (qq, kk, vv), up)
                    g["q"][qa + a:qa + b, hs] = gq
                    g["k"][ka + key, h] += gk
                    g["v"][ka + key, h] += gv
        qa, ka = qa + m, ka + room
    out = {"o": o.view(s["q"].shape),
           "lse": lse if case["form"] == "packed" else lse.view(H, case["B"], -1).transpose(0, 1).contiguous()}
    for x in g:
        out["d" + x] = g[x].view(s[x].shape)
    return out
