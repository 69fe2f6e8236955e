"""The operators around the 8-bit frame cache, as measured work.

qk_norm_rope, cache_write, cache_append, cache_read and forward_cache: listed and drawn
cases, their inputs, their plain forms (fp32 torch operations, rounded once at the end) and
their definitions in 64 bits.  The shapes are this repository's: 30x52-patch frames
(P = 1560), 12 heads of 128 elements, 3-frame chunks and caches of 6, 7 or 13 frames by head
role, next to generic ones (64-element heads, pages of 16 or 64 tokens, shared key heads).
"""
import math

import torch

own = False
BLOCK = 32                  # elements of a row that share one scale
E_MIN, E_MAX = -124, 119    # exponents a scale can take
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, B=1, H=12, Hkv=12, L=1, d=128, page=64, per_head=False, ragged=False,
             layout="interleaved", axes="44,42,42", far=False, kv=0, causal=False, roles=False, blhd=False)
    c.update(kw)
    return c


def listed():
    return [
        # one new token of eight sequences, half layout on half of the head, far positions
        _case("norm_rope token", "norm_rope", B=8, layout="half", axes="64", far=True),
        # a streaming chunk: 3 frames of 30x52 patches, three position axes
        _case("norm_rope chunk", "norm_rope", L=4680),
        # a whole 41-frame video as the projections leave it, [B, L, H, d] in memory
        _case("norm_rope video", "norm_rope", L=63960, blhd=True),
        # one frame into per-head frame slots
        _case("write frame", "write", L=1560, page=1560, per_head=True),
        # padded prompts of uneven length into 16-token pages
        _case("write prompts", "write", B=4, H=8, Hkv=4, L=1021, d=64, page=16, ragged=True),
        # one new token of sixteen sequences, shared key heads
        _case("append token", "append", B=16, Hkv=4, layout="half", axes="128", far=True),
        # the chunk of a streaming step into per-head frame slots
        _case("append chunk", "append", L=4680, page=1560, per_head=True),
        # the 13 frames of a memory head's cache, all heads, back as bf16
        _case("read frames", "read", L=20280, page=1560, per_head=True),
        # uneven windows out of 16-token pages
        _case("read windows", "read", B=3, H=4, Hkv=4, L=777, d=64, page=16, ragged=True),
        # one new token of eight sequences over long caches
        _case("attend token", "attend", B=8, kv=16384, ragged=True),
        # a causal chunk with shared key heads over 16-token pages
        _case("attend causal", "attend", B=2, Hkv=4, L=333, d=64, page=16, kv=4099, ragged=True, causal=True),
        # a streaming chunk over per-head caches of 6, 7 and 13 frames
        _case("attend stream", "attend", L=4680, page=1560, per_head=True, kv=20280, roles=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "write", "append", "read", "attend", "attend"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 12])
    h = hkv * rng.choice([1, 1, 2, 3])
    b = _log(rng, 1, 16)
    c = _case("", op, B=b, H=h, Hkv=hkv, d=d, page=rng.choice([16, 40, 64, 200, 1560]), ragged=rng.random() < 0.5,
              per_head=rng.random() < 0.5, blhd=rng.random() < 0.5, far=rng.random() < 0.5)
    del c["name"]
    c["layout"] = rng.choice(["interleaved", "half"])
    if c["layout"] == "half":
        c["axes"] = rng.choice(["64", "32", "16,24,24"] + (["128", "32,48,48", "96"] if d == 128 else ["48"]))
    else:
        c["axes"] = rng.choice(["64", "22", "24,20,20"] + (["128", "44,42,42", "90"] if d == 128 else ["10,10,10"]))
    if op == "attend":
        c["L"] = _log(rng, 1, 4680)
        c["kv"] = max(1, min(_log(rng, 16, 20280), int(8e8 / (b * h * c["L"]))))
        c["causal"] = rng.random() < 0.5
        if c["causal"]:
            c["kv"] = max(c["kv"], min(c["L"], int(8e8 / (b * h * c["L"]))))
    else:
        c["L"] = _log(rng, 1, max(2, 400000 // (b * h)))
    return c


def _lens(c, full):
    """[B][Hkv] lengths that the case stands for, from the case alone."""
    if c["roles"]:  # local, anchor and memory heads keep 6, 7 and 13 frames
        return [[min(full, (6, 7, 13)[3 * h // c["Hkv"]] * c["page"]) for h in range(c["Hkv"])] for _ in range(c["B"])]
    if not c["ragged"]:
        return [[full] * c["Hkv"] for _ in range(c["B"])]
    per_head = c["per_head"] and c["op"] == "attend"
    return [[full - ((b * 5 + (h if per_head else 0) * 3) * full // 17) % (full // 2 + 1) for h in range(c["Hkv"])]
            for b in range(c["B"])]


def work(c):
    B, H, Hk, L, d = c["B"], c["H"], c["Hkv"], c["L"], c["d"]
    row = d + d // BLOCK
    if c["op"] == "norm_rope":
        n_ax = len(c["axes"].split(","))
        return {"bytes": 4.0 * B * (H + Hk) * L * d + 4.0 * B * L * n_ax, "flops": 8.0 * B * (H + Hk) * L * d}
    if c["op"] == "attend":
        by, fl = 4.0 * B * H * L * d + 4.0 * B * H * L, 0.0
        for b, lens in enumerate(_lens(c, c["kv"])):
            for n in lens:
                by += 2.0 * n * row
                pairs = L * n
                if c["causal"]:  # query i sees n - L + i + 1 keys, none where that is negative
                    first = max(0, L - n)
                    pairs = (L - first) * (n - L + first + 1 + n) // 2
                fl += 4.0 * d * pairs * (H // Hk)
        return {"bytes": by, "flops": fl}
    tok = sum(lens[0] for lens in _lens(c, L))
    if c["op"] == "append":
        return {"bytes": tok * (4.0 * H * d + Hk * (4.0 * d + 2.0 * row)), "flops": 10.0 * tok * (H + 2 * Hk) * d}
    return {"bytes": tok * Hk * (4.0 * d + 2.0 * row), "flops": 4.0 * tok * Hk * d}


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _tensor(g, c, heads, L):
    """bf16 [B, heads, L, d], in memory as [B, L, heads, d] where the case says so."""
    if c["blhd"]:
        return _randn(g, c["B"], L, heads, c["d"]).bfloat16().transpose(1, 2)
    return _randn(g, c["B"], heads, L, c["d"]).bfloat16()


def _empty_like(t):
    return torch.zeros_like(t)


def _quantise(x):
    """fp32 [..., d] -> (e4m3 codes, E8M0 scales [..., d / 32])."""
    blk = x.unflatten(-1, (x.shape[-1] // BLOCK, BLOCK))
    mant, ex = torch.frexp(blk.abs().amax(-1))
    e = (ex - 9 + (mant > 0.875).int()).clamp(E_MIN, E_MAX)
    e = torch.where(mant == 0, torch.full_like(e, E_MIN), e)
    codes = torch.ldexp(blk, -e.unsqueeze(-1)).clamp(-448.0, 448.0).flatten(-2).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _inv_freq(c):
    """Inverse frequencies (64 bits) of every pair, per axis, base 10000; far positions interpolate by 4."""
    f = [10000.0 ** (-2.0 * i / n) for n in map(int, c["axes"].split(",")) for i in range(n // 2)]
    return torch.tensor(f, dtype=torch.float64, device=DEV) / (4.0 if c["far"] else 1.0)


def _positions(g, c, axes):
    """int32 [B, L, axes]: frame, row and column of a 30x52 grid, or token numbers."""
    B, L, n = c["B"], c["L"], len(axes)
    base = torch.randint(0, 1 << 20 if c["far"] else 1 << 10, (B, 1), generator=g, device=DEV)
    i = torch.arange(L, device=DEV).unsqueeze(0)
    if n == 1:
        return (base + i).to(torch.int32).unsqueeze(-1).contiguous()
    return torch.stack([base + i // 1560, (i // 52 % 30).expand(B, L), (i % 52).expand(B, L)], -1).to(torch.int32).contiguous()


def _pool(g, c, tokens, random_codes):
    """A page pool, the page table int32 [B, Hkv or 1, N] and the pool's head count."""
    P = c["page"]
    n = -(-tokens // P)
    rows = c["Hkv"] if c["per_head"] else 1
    heads = 1 if c["per_head"] else c["Hkv"]
    n_pages = c["B"] * rows * n + 3
    table = torch.randperm(n_pages, generator=g, device=DEV)[: c["B"] * rows * n].to(torch.int32)
    s = {"table": table.reshape(c["B"], rows, n).contiguous(), "heads": heads}
    for name in ("k", "v"):
        if random_codes:
            x = _randn(g, n_pages, heads, P, c["d"]) * torch.exp(0.5 * _randn(g, n_pages, heads, P, 1))
            s[name + "_codes"], s[name + "_scale"] = _quantise(x)
        else:
            s[name + "_codes"] = torch.zeros(n_pages, heads, P, c["d"], device=DEV).to(torch.float8_e4m3fn)
            s[name + "_scale"] = torch.ones(n_pages, heads, P, c["d"] // BLOCK, device=DEV).to(torch.float8_e8m0fnu)
    return s


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, B, H, Hk, L, d = c["op"], c["B"], c["H"], c["Hkv"], c["L"], c["d"]
    s = {"case": c}
    if op in ("norm_rope", "append"):
        axes = [int(n) for n in c["axes"].split(",")]
        s["pairs"] = tuple(n // 2 for n in axes)
        s["inv_freq"] = _inv_freq(c)
        s["rope_scale"] = 0.1 * math.log(4.0) + 1.0 if c["far"] else 1.0
        s["pos"] = _positions(g, c, axes)
        s["q"], s["k"] = _tensor(g, c, H, L), _tensor(g, c, Hk, L)
        s["qw"], s["kw"] = 1.0 + 0.1 * _randn(g, d), 1.0 + 0.1 * _randn(g, d)
        s["q_out"] = _empty_like(s["q"])
        if op == "norm_rope":
            s["k_out"] = _empty_like(s["k"])
            return s
    if op in ("write", "append"):
        # each sequence's tokens go behind what its cache holds already
        start = torch.randint(0, c["page"], (B,), generator=g, device=DEV)
        s.update(_pool(g, c, L + c["page"], False))
        s["start"] = start.to(torch.int32)
        if op == "write":
            s["k"] = _tensor(g, c, Hk, L)
        s["v"] = _tensor(g, c, Hk, L)
        s["lens"] = torch.tensor([x[0] for x in _lens(c, L)], dtype=torch.int32, device=DEV)
    elif op == "read":
        s.update(_pool(g, c, L + c["page"], True))
        s["start"] = torch.randint(0, c["page"], (B,), generator=g, device=DEV).to(torch.int32)
        s["lens"] = torch.tensor([x[0] for x in _lens(c, L)], dtype=torch.int32, device=DEV)
        s["k_out"] = torch.zeros(B, Hk, L, d, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.zeros_like(s["k_out"])
    elif op == "attend":
        s.update(_pool(g, c, c["kv"], True))
        s["q"] = _tensor(g, c, H, L)
        s["kv_lens"] = torch.tensor(_lens(c, c["kv"]), dtype=torch.int32, device=DEV)
        s["out"] = _empty_like(s["q"])
        s["lse"] = torch.zeros(B, H, L, dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------ the plain forms
def _norm_rope(x, w, s):
    """fp32 [B, heads, L, d]: the norm of every head's row, then the rotation of its first elements."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    axis = torch.repeat_interleave(torch.arange(len(s["pairs"]), device=DEV), torch.tensor(s["pairs"], device=DEV))
    angle = s["pos"].double()[..., axis] * s["inv_freq"]
    cos = (torch.cos(angle) * s["rope_scale"]).float().unsqueeze(1)
    sin = (torch.sin(angle) * s["rope_scale"]).float().unsqueeze(1)
    R = 2 * sum(s["pairs"])
    if s["case"]["layout"] == "half":
        a, b = x[..., : R // 2], x[..., R // 2: R]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., R:]], -1)


def _rows(s, tokens):
    """Pool rows [B, Hkv, tokens] of the tokens behind `start`, and which of them are there."""
    c, P = s["case"], s["case"]["page"]
    i = torch.arange(tokens, device=DEV)
    pos = s["start"].long()[:, None] + i
    page = s["table"].long().expand(-1, c["Hkv"], -1).gather(2, (pos // P).unsqueeze(1).expand(-1, c["Hkv"], -1))
    head = torch.arange(c["Hkv"], device=DEV)[None, :, None] if s["heads"] > 1 else 0
    there = (i < s["lens"].long()[:, None]).unsqueeze(1).expand(-1, c["Hkv"], -1)
    return (page * s["heads"] + head) * P + (pos % P).unsqueeze(1), there


def _store(s, name, x, rows, there):
    codes, scale = _quantise(x)
    d = s["case"]["d"]
    s[name + "_codes"].view(torch.uint8).view(-1, d)[rows[there]] = codes.view(torch.uint8)[there]
    s[name + "_scale"].view(torch.uint8).view(-1, d // BLOCK)[rows[there]] = scale.view(torch.uint8)[there]


def _value(s, name, rows):
    """fp32 values of the pool's rows."""
    d = s["case"]["d"]
    codes = s[name + "_codes"].view(torch.uint8).view(-1, d)[rows].view(torch.float8_e4m3fn).float()
    scale = s[name + "_scale"].view(torch.uint8).view(-1, d // BLOCK)[rows].view(torch.float8_e8m0fnu).float()
    return codes * scale.repeat_interleave(BLOCK, -1)


def _pools(s):
    return s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]


def _attend(s):
    c = s["case"]
    B, H, Hk, L, d, N, P = c["B"], c["H"], c["Hkv"], c["L"], c["d"], c["kv"], c["page"]
    i = torch.arange(N, device=DEV)
    page = s["table"].long()[..., i // P].expand(-1, Hk, -1)
    head = torch.arange(Hk, device=DEV)[None, :, None] if s["heads"] > 1 else 0
    rows = (page * s["heads"] + head) * P + i % P
    seen = i < s["kv_lens"].long().unsqueeze(-1)
    k = torch.where(seen.unsqueeze(-1), _value(s, "k", rows), 0.0)
    v = torch.where(seen.unsqueeze(-1), _value(s, "v", rows), 0.0)
    q = s["q"].float().reshape(B, Hk, H // Hk, L, d)
    x = (q @ k.transpose(-1, -2).unsqueeze(2)) * (1.0 / math.sqrt(d))
    seen = seen[:, :, None, None, :]
    if c["causal"]:
        last = s["kv_lens"].long()[:, :, None, None, None] - L + torch.arange(L, device=DEV)[:, None]
        seen = seen & (i <= last)
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = x.sum(-1, keepdim=True)
    o = (x @ v.unsqueeze(2)) / torch.where(total == 0, 1.0, total)
    s["out"].copy_(o.reshape(B, H, L, d))
    s["lse"].copy_((m + torch.log(total)).reshape(B, H, L))
    return s["out"], s["lse"]


def _run_own(s):
    import frame_sparse_attention_b200 as sfa
    c = s["case"]
    op = c["op"]
    if op in ("norm_rope", "append"):
        rope = sfa.RopeTable(s["inv_freq"], s["pairs"], s["rope_scale"])
    if op == "norm_rope":
        return sfa.qk_norm_rope(s["q"], s["k"], rope=rope, positions=s["pos"], q_weight=s["qw"], k_weight=s["kw"],
                                eps=EPS, layout=c["layout"], q_out=s["q_out"], k_out=s["k_out"])
    cache = sfa.FrameCache(s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])
    if op == "write":
        sfa.cache_write(cache, s["k"], s["v"], s["table"], s["start"], lens=s["lens"])
        return _pools(s)
    if op == "append":
        q = sfa.cache_append(cache, s["q"], s["k"], s["v"], s["table"], s["start"], lens=s["lens"], rope=rope,
                             positions=s["pos"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, layout=c["layout"],
                             q_out=s["q_out"])
        return (q,) + _pools(s)
    if op == "read":
        return sfa.cache_read(cache, s["table"], s["start"], c["L"], lens=s["lens"], k_out=s["k_out"], v_out=s["v_out"])
    return sfa.forward_cache(s["q"], cache, s["table"], s["kv_lens"], max_kv=c["kv"], causal=c["causal"], out=s["out"],
                             lse=s["lse"])


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "attend":
        return _attend(s)
    if op == "norm_rope":
        s["q_out"].copy_(_norm_rope(s["q"], s["qw"], s))
        s["k_out"].copy_(_norm_rope(s["k"], s["kw"], s))
        return s["q_out"], s["k_out"]
    rows, there = _rows(s, s["case"]["L"])
    if op == "read":
        s["k_out"].copy_(torch.where(there.unsqueeze(-1), _value(s, "k", rows), s["k_out"].float()))
        s["v_out"].copy_(torch.where(there.unsqueeze(-1), _value(s, "v", rows), s["v_out"].float()))
        return s["k_out"], s["v_out"]
    if op == "write":
        _store(s, "k", s["k"].float(), rows, there)
    else:
        # rows behind a sequence's length stay as they were; the cache takes the key as a bf16 value
        q_there = (torch.arange(s["q"].shape[2], device=DEV) < s["lens"].long()[:, None])[:, None, :, None]
        s["q_out"].copy_(torch.where(q_there, _norm_rope(s["q"], s["qw"], s), s["q_out"].float()))
        _store(s, "k", _norm_rope(s["k"], s["kw"], s).bfloat16().float(), rows, there)
    _store(s, "v", s["v"].float(), rows, there)
    return ((s["q_out"],) if op == "append" else ()) + _pools(s)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rows(x, w, s):
    """The norm and the rotation, pair by pair."""
    x = x.double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    half, p = s["case"]["layout"] == "half", 0
    out, R = y.clone(), 2 * sum(s["pairs"])
    for axis, n in enumerate(s["pairs"]):
        for _ in range(n):
            i, j = (p, p + R // 2) if half else (2 * p, 2 * p + 1)
            t = (s["pos"][:, None, :, axis].double() * s["inv_freq"][p])
            out[..., i] = s["rope_scale"] * (y[..., i] * torch.cos(t) - y[..., j] * torch.sin(t))
            out[..., j] = s["rope_scale"] * (y[..., j] * torch.cos(t) + y[..., i] * torch.sin(t))
            p += 1
    return out


def _exact_block(x):
    """(code values, scales) of 64-bit rows: the smallest power of two that brings a block within 448, and the
    nearest e4m3 values (4 significant bits, steps of 2^-9 at least), ties to even."""
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -140) / 448.0))
    e = torch.where(top > 448.0 * 2.0 ** e, e + 1, e)  # the logarithm's own rounding
    e = torch.where(top <= 448.0 * 2.0 ** (e - 1), e - 1, e).clamp(E_MIN, E_MAX)
    y = (b * 2.0 ** -e).clamp(-448.0, 448.0)
    _, ex = torch.frexp(y)
    step = 2.0 ** torch.clamp(ex.double() - 4, min=-9.0)
    return (torch.round(y / step) * step).flatten(-2), (2.0 ** e).squeeze(-1)


def _exact_place(s, b, h, i):
    """(page, head of the pool, row of the page) of token i of sequence b and key head h."""
    P = s["case"]["page"]
    t = s["table"][b, h if s["table"].shape[1] > 1 else 0].long()
    return t[i // P], (h if s["heads"] > 1 else 0), i % P


def _exact_attend(s):
    c = s["case"]
    L, d = c["L"], c["d"]
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        for h in range(c["H"]):
            hk = h * c["Hkv"] // c["H"]
            n = int(s["kv_lens"][b, hk])
            at = _exact_place(s, b, hk, torch.arange(n, device=DEV))
            k, v = ((s[x + "_codes"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double().unflatten(-1, (-1, BLOCK))
                     * s[x + "_scale"].view(torch.uint8)[at].view(torch.float8_e8m0fnu).double().unsqueeze(-1)).flatten(-2)
                    for x in ("k", "v"))
            t = torch.einsum("id,jd->ij", s["q"][b, h].double(), k) / math.sqrt(d)
            if c["causal"]:
                hidden = torch.arange(n, device=DEV)[None, :] > n - L + torch.arange(L, device=DEV)[:, None]
                t = t.masked_fill(hidden, -math.inf)
            lse[b, h] = torch.logsumexp(t, -1)
            o[b, h] = torch.nan_to_num(torch.exp(t - lse[b, h][:, None]), nan=0.0) @ v
    return o, lse


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "attend":
        return _exact_attend(s)
    if op == "norm_rope":
        return _exact_rows(s["q"], s["qw"], s), _exact_rows(s["k"], s["kw"], s)
    if op == "read":
        out = [s["k_out"].double(), s["v_out"].double()]
    else:
        k = s["k"].double() if op == "write" else _exact_rows(s["k"], s["kw"], s).bfloat16().double()
        new = {"k": _exact_block(k), "v": _exact_block(s["v"].double())}
        out = {x: s[x].double() for x in ("k_codes", "k_scale", "v_codes", "v_scale")}
    for b in range(c["B"]):
        m = int(s["lens"][b])
        for h in range(c["Hkv"]):
            at = _exact_place(s, b, h, int(s["start"][b]) + torch.arange(m, device=DEV))
            for j, x in enumerate(("k", "v")):
                if op == "read":
                    blk = s[x + "_codes"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double().unflatten(-1, (-1, BLOCK))
                    sc = s[x + "_scale"].view(torch.uint8)[at].view(torch.float8_e8m0fnu).double()
                    out[j][b, h, :m] = (blk * sc.unsqueeze(-1)).flatten(-2)
                else:
                    out[x + "_codes"][at] = new[x][0][b, h, :m]
                    out[x + "_scale"][at] = new[x][1][b, h, :m]
    if op == "read":
        return tuple(out)
    pools = tuple(out[x] for x in ("k_codes", "k_scale", "v_codes", "v_scale"))
    if op == "write":
        return pools
    q = s["q_out"].double()
    rows = _exact_rows(s["q"], s["qw"], s)
    for b in range(c["B"]):
        q[b, :, : int(s["lens"][b])] = rows[b, :, : int(s["lens"][b])]
    return (q,) + pools
