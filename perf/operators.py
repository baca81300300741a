"""Measured cases of the attention operators over a 4-bit key/value cache.

Three operators of the serving step between the QKV product and the output product:

* ``norm_rope``: RMS norm of every query and key head and the position rotation, one pass over the fused rows;
* ``append``: the same for the queries and keys of new tokens, with the keys and values stored into a paged
  4-bit cache on the way, and the stored values read back;
* ``attn``: attention of the queries over that cache, single tokens and chunks.

Cache block (16 tokens of one key/value head, D channels, G = D/32 scale groups; Gp = 4 if G % 4 == 0 else G, and
G/Gp planes), in this order:

* key nibbles   [plane][row 16][c 4][group Gp] 32-bit words; word nibble i is channel 32*group + 8*c + i, and row
  8*h + 2*a + b holds token 4*a + 2*h + b;
* value nibbles [plane][u 2][r 8][c 4][group Gp] 32-bit words; nibble 4*b + j is channel 32*group + 4*r + j of token
  4*c + 2*u + b;
* key scales    [token 16][G] fp16;
* value scales  [token 16][G] fp16.

A value is scale * (nibble - 8).  The scale of 32 values is the fp16 of (the value of largest magnitude, the positive
one of a tie) / -8, and a nibble is floor(x / scale + 8.5) held to 0..15 (8 where the scale is 0).

A cache is a uint8 tensor [pages][kv heads][blocks a page][18 * D]; slot s is token s % page of page s // page.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a model of 32 query and 8 key heads of 128 channels: latency only
        dict(name="rope_1tok", op="norm_rope", tokens=1, nq=32, nk=8, D=128, rot=128, dtype="f32", norm=True,
             interleaved=False, n_pos=8192),
        # a prompt chunk of the prefill GEMM's size, rotation of neighbouring pairs, no norm
        dict(name="rope_512tok_pairs", op="norm_rope", tokens=512, nq=32, nk=8, D=128, rot=128, dtype="f32",
             norm=False, interleaved=True, n_pos=8192),
        # a long prompt in 16 bits, heads of 96 channels of which 72 rotate, a position table for long contexts
        dict(name="rope_8191tok_96", op="norm_rope", tokens=8191, nq=32, nk=32, D=96, rot=72, dtype="bf16", norm=True,
             interleaved=False, n_pos=131072),
        # decode of one sequence: norm, rotation and append of one token
        dict(name="append_1tok", op="append", batch=1, new=1, nq=32, nkv=8, D=128, rot=128, page=16, dtype="f32",
             norm=True, interleaved=False, n_pos=8192),
        # decode of 64 sequences, the head layout of the 896-wide model (14 query, 2 key heads of 64)
        dict(name="append_64seq", op="append", batch=64, new=1, nq=14, nkv=2, D=64, rot=64, page=64, dtype="f16",
             norm=False, interleaved=False, n_pos=32768),
        # prompt chunks of four sequences, 16-bit activations
        dict(name="append_4x2048", op="append", batch=4, new=2048, nq=32, nkv=8, D=128, rot=128, page=64,
             dtype="bf16", norm=True, interleaved=True, n_pos=32768),
        # the first tokens of a reply in the 576-wide model (9 query, 3 key heads of 64): latency only
        dict(name="attn_short", op="attn", batch=1, new=1, max_len=37, ragged=False, nq=9, nkv=3, D=64, page=16,
             window=0, dtype="f32"),
        # one sequence, long context, fp32 activations as the GEMVs use them
        dict(name="attn_1x32768", op="attn", batch=1, new=1, max_len=32768, ragged=False, nq=32, nkv=8, D=128,
             page=64, window=0, dtype="f32"),
        # 16 sequences of uneven odd lengths, 7 query heads a key head, fp32
        dict(name="attn_16x9001_ragged", op="attn", batch=16, new=1, max_len=9001, ragged=True, nq=14, nkv=2, D=64,
             page=16, window=0, dtype="f32"),
        # a full decode batch in 16 bits
        dict(name="attn_64x8192", op="attn", batch=64, new=1, max_len=8192, ragged=False, nq=32, nkv=8, D=128,
             page=64, window=0, dtype="bf16"),
        # chunked prefill in chunks of 64 positions beside decoding sequences, sliding window
        dict(name="attn_mixed_64", op="attn", batch=8, new=64, max_len=5000, ragged=True, nq=32, nkv=8, D=128,
             page=32, window=4096, dtype="f32"),
        # a prompt chunk of 1024 tokens at the end of a 16384-token context
        dict(name="attn_chunk_1024", op="attn", batch=1, new=1024, max_len=16384, ragged=False, nq=32, nkv=8, D=128,
             page=64, window=0, dtype="bf16"),
    ]


# (query heads, key/value heads, head size)
HEADS = [(9, 3, 64), (14, 2, 64), (32, 8, 128), (32, 32, 96), (8, 1, 256), (24, 2, 128), (16, 16, 64), (28, 4, 128)]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attn", "attn"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    nq, nkv, D = rng.choice(HEADS)
    if op == "norm_rope":
        return dict(op=op, tokens=_log_int(rng, 1, 4000), nq=nq, nk=nkv, D=D, rot=rng.choice([D, D, D // 2, 3 * D // 4]),
                    dtype=dtype, norm=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    n_pos=rng.choice([8192, 32768, 131072]))
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "append":
        new = _log_int(rng, 1, 2048)
        batch = _log_int(rng, 1, max(1, min(128, 4000 // new)))
        return dict(op=op, batch=batch, new=new, nq=nq, nkv=nkv, D=D, rot=rng.choice([D, D, D // 2, 3 * D // 4]),
                    page=page, dtype=dtype, norm=rng.random() < 0.5, interleaved=rng.random() < 0.5, n_pos=32768)
    chunk = rng.random() < 0.4
    max_len = _log_int(rng, 1, 32768)
    # at most the cache bytes of the largest listed decode and the products of the largest listed chunk
    room = 250_000_000 // max(1, max_len * nkv * 18 * D // 16)
    new = min(_log_int(rng, 2, 1024), max_len) if chunk else 1
    if chunk:
        new = max(1, min(new, int(2e11 / (4.0 * max_len * nq * D))))
        room = min(room, int(2e11 / (4.0 * max_len * new * nq * D)))
    batch = _log_int(rng, 1, max(1, min(64, room)))
    return dict(op=op, batch=batch, new=new, max_len=max_len, ragged=rng.random() < 0.6, nq=nq, nkv=nkv, D=D,
                page=page, window=rng.choice([0, 0, 0, 1024, 100]), dtype=dtype)


def _lens(case):
    """Lengths and new tokens of each sequence: the first has both at their largest."""
    B, L, n = case["batch"], case["max_len"], case["new"]
    if not case["ragged"]:
        return [L] * B, [n] * B
    part = [1.0 if b == 0 else (b * 0.6180339887498949) % 1.0 for b in range(B)]
    new = [n if b % 3 == 0 else 1 for b in range(B)]
    return [max(new[b], int(L * part[b])) for b in range(B)], new


def _seen(length, new, window):
    """Keys that the `new` last positions of a sequence see, summed."""
    total = 0
    for i in range(new):
        k = length - new + i + 1
        total += min(k, window) if window else k
    return total


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    nq, D = case["nq"], case["D"]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (nq + case["nk"]) * D
        return dict(bytes=2 * size * n + case["tokens"] * (4 + 4 * case["rot"]), flops=10 * n)
    nkv = case["nkv"]
    if case["op"] == "append":
        T = case["batch"] * case["new"]
        # q in and out, k and v in, the cache rows written and read once, their values out in fp16
        n = T * (2 * nq * D * size + 2 * nkv * D * size + 2 * nkv * 18 * D // 16 + 2 * nkv * D * 2)
        return dict(bytes=n + T * (4 + 8 + 4 * case["rot"]), flops=10 * T * (nq + 2 * nkv) * D)
    lens, new = _lens(case)
    w = case["window"]
    keys = sum(min(l, w + n - 1) if w else l for l, n in zip(lens, new))
    seen = sum(_seen(l, n, w) for l, n in zip(lens, new))
    return dict(bytes=keys * nkv * 18 * D // 16 + 2 * sum(new) * nq * D * size, flops=4 * seen * nq * D)


# ---------------------------------------------------------------- inputs

def _table(n_pos, rot, device):
    """cos and sin of position * 10000^(-2i/rot), computed in 64 bits: [n_pos][rot/2][2] fp32."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    a = torch.arange(n_pos, device=device, dtype=torch.float64)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float()


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dt, D, nq = DT[case["dtype"]], case["D"], case["nq"]
    if case["op"] == "norm_rope":
        T, nk = case["tokens"], case["nk"]
        s["x"] = _normal(g, T, (nq + nk) * D).to(dt)
        s["positions"] = torch.randint(0, case["n_pos"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["table"] = _table(case["n_pos"], case["rot"], "cuda")
        s["q_weight"] = 1 + _normal(g, D, scale=0.2) if case["norm"] else None
        s["k_weight"] = 1 + _normal(g, D, scale=0.2) if case["norm"] else None
        return s
    nkv, page = case["nkv"], case["page"]
    if case["op"] == "append":
        B, n = case["batch"], case["new"]
        T = B * n
        # one fused row a token, as the QKV product writes it
        s["qkv"] = _normal(g, T, (nq + 2 * nkv) * D).to(dt)
        past = torch.randint(0, case["n_pos"] - n, (B, 1), generator=g, device="cuda")
        i = torch.arange(n, device="cuda")
        s["positions"] = (past + i).reshape(-1).int()
        per = (n + page - 2) // page + 1
        pages = torch.randperm(B * per + 3, generator=g, device="cuda")[:B * per].reshape(B, per)
        at = past % page + i
        s["slots"] = (pages.gather(1, at // page) * page + at % page).reshape(-1)
        s["table"] = _table(case["n_pos"], case["rot"], "cuda")
        s["q_weight"] = 1 + _normal(g, D, scale=0.2) if case["norm"] else None
        s["k_weight"] = 1 + _normal(g, D, scale=0.2) if case["norm"] else None
        s["cache"] = torch.zeros(B * per + 3, nkv, page // 16, 18 * D, dtype=torch.uint8, device="cuda")
        return s
    lens, new = _lens(case)
    B, T = case["batch"], sum(new)
    need = [-(-l // page) for l in lens]
    width, total = max(need), sum(need)
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    cache = torch.empty(total, nkv, page // 16, 18 * D, dtype=torch.uint8, device="cuda")
    spread = _normal(g, nkv, 1, D, scale=0.5).exp()      # a few key channels are much larger than others
    step = max(1, (1 << 26) // (nkv * page * D))
    for p in range(0, total, step):
        m = min(step, total - p)
        k = _normal(g, m, nkv, page, D) * spread
        v = _normal(g, m, nkv, page, D)
        cache[p:p + m] = _pack(*_quantise(k), *_quantise(v))
    s["cache"], s["page_table"] = cache, table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda") if case["new"] > 1 else None
    s["q"] = _normal(g, T, nq * D, scale=1.5).to(dt)
    s["out"] = torch.empty(T, nq * D, dtype=dt, device="cuda")
    # scratch of a serving loop, kept between calls (zeroed once)
    s["workspace"] = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- the cache format, in torch

def _quantise(x):
    """x [..., D] fp32 -> nibbles [..., D] uint8 and scales [..., D/32] fp16."""
    b = x.unflatten(-1, (-1, 32))
    hi, lo = b.amax(-1), b.amin(-1)
    d = (torch.where(hi >= -lo, hi, lo) / -8).half()
    n = (b / d.float()[..., None] + 8.5).floor().clamp(0, 15)
    return torch.where(d[..., None] != 0, n, torch.full_like(n, 8)).flatten(-2).to(torch.uint8), d


def _planes(D):
    G = D // 32
    Gp = 4 if G % 4 == 0 else G
    return G // Gp, Gp


def _pack(kn, kd, vn, vd):
    """Nibbles [..., page, D] and scales [..., page, G] of keys and values -> blocks [..., page/16, 18 D]."""
    *lead, page, D = kn.shape
    pl, Gp = _planes(D)
    k = kn.reshape(-1, 4, 2, 2, pl, Gp, 4, 8).permute(0, 4, 2, 1, 3, 6, 5, 7)     # plane, h, a, b, c, group, i
    v = vn.reshape(-1, 4, 2, 2, pl, Gp, 8, 4).permute(0, 4, 2, 6, 1, 5, 3, 7)     # plane, u, r, c, group, b, j
    parts = []
    for n in (k, v):
        n = n.reshape(n.shape[0], -1, 2)
        parts.append(n[..., 0] | (n[..., 1] << 4))
    for d in (kd, vd):
        parts.append(d.reshape(parts[0].shape[0], -1).contiguous().view(torch.uint8))
    return torch.cat(parts, -1).reshape(*lead, page // 16, 18 * D)


def _unpack(blocks):
    """Blocks [..., 18 D] -> keys and values [..., 16, D] fp32."""
    *lead, size = blocks.shape
    D = size // 18
    G = D // 32
    pl, Gp = _planes(D)
    b = blocks.reshape(-1, size)
    out = []
    for at, shape, order in ((0, (pl, 2, 4, 2, 4, Gp, 8), (0, 3, 2, 4, 1, 6, 5, 7)),
                             (8 * D, (pl, 2, 8, 4, Gp, 2, 4), (0, 4, 2, 6, 1, 5, 3, 7))):
        n = b[:, at:at + 8 * D]
        n = torch.stack([n & 15, n >> 4], -1).reshape(-1, *shape).permute(*order).reshape(-1, 16, G, 32)
        d = b[:, 16 * D + (at // 8):16 * D + (at // 8) + D].contiguous().view(torch.float16).reshape(-1, 16, G, 1)
        out.append(((n.float() - 8) * d.float()).reshape(*lead, 16, D))
    return out


# ---------------------------------------------------------------- one pass

def run(s):
    return {"norm_rope": _run_rope, "append": _run_append, "attn": _run_attn}[s["op"]](s)


def _norm_rope(x, weight, positions, table, interleaved, eps=1e-6):
    """x [T][heads][D] fp32: RMS norm with weight (None: no norm), then rotation of the first 2 * table.shape[1]
    channels."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    cs = table[positions.long()]
    c, n = cs[:, None, :, 0], cs[:, None, :, 1]
    half = table.shape[1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, v = a * c - b * n, a * n + b * c
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1)


def _run_rope(s):
    x, nq, nk, D = s["x"], s["nq"], s["nk"], s["D"]
    if own:
        from quantised_gguf_weight_gb300 import qk
        return qk.norm_rope(x, nq, nk, D, s["positions"], s["table"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                            eps=1e-6, interleaved=s["interleaved"])
    h = x.float().reshape(x.shape[0], nq + nk, D)
    q = _norm_rope(h[:, :nq], s["q_weight"], s["positions"], s["table"], s["interleaved"])
    k = _norm_rope(h[:, nq:], s["k_weight"], s["positions"], s["table"], s["interleaved"])
    return torch.cat([q, k], 1).reshape(x.shape).to(x.dtype)


def _run_append(s):
    nq, nkv, D, cache = s["nq"], s["nkv"], s["D"], s["cache"]
    q, k, v = s["qkv"].split([nq * D, nkv * D, nkv * D], 1)
    if own:
        from quantised_gguf_weight_gb300 import qk
        qo = qk.kv_append_q4(cache, q, k, v, s["positions"], s["slots"], s["table"], q_weight=s["q_weight"],
                             k_weight=s["k_weight"], eps=1e-6, interleaved=s["interleaved"])
        kc, vc = qk.kv_read_q4(cache, s["slots"], dtype=torch.float16)
        return {"q": qo, "k": kc, "v": vc}
    T = q.shape[0]
    qo = _norm_rope(q.float().reshape(T, nq, D), s["q_weight"], s["positions"], s["table"], s["interleaved"])
    ko = _norm_rope(k.float().reshape(T, nkv, D), s["k_weight"], s["positions"], s["table"], s["interleaved"])
    (kn, kd), (vn, vd) = _quantise(ko), _quantise(v.float().reshape(T, nkv, D))
    # bytes of a token inside its block: nibble bytes hold two channels of one token
    block = cache.reshape(cache.shape[0], nkv, -1)
    page = 16 * cache.shape[2]
    p, t = s["slots"] // page, s["slots"] % page
    kb, vb = _token_bytes(t, D)
    head = torch.arange(nkv, device=cache.device)[:, None]
    where = lambda o: (p[:, None, None], head, o[:, None, :])  # noqa: E731
    kn, vn = kn.reshape(T, nkv, -1, 2), vn.reshape(T, nkv, -1, 2)
    block[where(kb[0])] = kn[..., 0] | (kn[..., 1] << 4)
    block[where(vb[0])] = vn[..., 0] | (vn[..., 1] << 4)
    block[where(kb[1])] = kd.contiguous().view(torch.uint8)
    block[where(vb[1])] = vd.contiguous().view(torch.uint8)
    # read back
    kc, vc = [], []
    for got, (no, so) in ((kc, kb), (vc, vb)):
        n = block[where(no)]
        n = torch.stack([n & 15, n >> 4], -1).reshape(T, nkv, -1, 32)
        d = block[where(so)].contiguous().view(torch.float16)
        got.append(((n.float() - 8) * d.float()[..., None]).reshape(T, nkv * D).half())
    return {"q": qo.reshape(T, nq * D).to(s["qkv"].dtype), "k": kc[0], "v": vc[0]}


def _token_bytes(t, D):
    """Byte offsets in a page's head of token t's key nibbles (channel pairs in order) and scales, and its value's."""
    G = D // 32
    pl, Gp = _planes(D)
    dev = t.device
    base, t = (t // 16 * 18 * D)[:, None], (t % 16)[:, None]
    ch = torch.arange(0, D, 2, device=dev)
    g = ch // 32
    plane, gp = g // Gp, g % Gp
    row = 8 * (t // 2 % 2) + 2 * (t // 4) + t % 2
    kb = ((plane * 16 + row) * 4 + ch % 32 // 8) * Gp + gp
    kb = base + 4 * kb + ch % 8 // 2
    vb = (((plane * 2 + t // 2 % 2) * 8 + ch % 32 // 4) * 4 + t // 4) * Gp + gp
    vb = base + 8 * D + 4 * vb + 2 * (t % 2) + ch % 4 // 2
    sc = torch.arange(2 * G, device=dev)
    ks = base + 16 * D + t * 2 * G + sc
    return (kb, ks), (vb, ks + D)


def _run_attn(s):
    q, nq, nkv, D = s["q"], s["nq"], s["nkv"], s["D"]
    scale = 1.0 / math.sqrt(D)
    if own:
        from quantised_gguf_weight_gb300 import qk
        return qk.attn_q4(s["cache"], q, s["page_table"], s["lens"], q_start=s["q_start"], max_q=s["new"],
                          max_len=s["max_len"], scale=scale, window=s["window"], out=s["out"],
                          workspace=s["workspace"])
    B, n, T = s["batch"], s["new"], q.shape[0]
    lens = s["lens"].long()
    start = s["q_start"].long() if s["q_start"] is not None else torch.arange(B + 1, device=q.device)
    count = start[1:] - start[:-1]
    i = torch.arange(n, device=q.device)
    rows = (start[:-1, None] + i).clamp(max=T - 1)
    x = q.float()[rows].reshape(B, n, nkv, nq // nkv, D).permute(0, 2, 3, 1, 4).reshape(B, nkv, -1, D)
    k, v = _unpack(s["cache"][s["page_table"].clamp(min=0).long()].transpose(1, 2))
    k, v = k.reshape(B, nkv, -1, D), v.reshape(B, nkv, -1, D)
    sc = torch.matmul(x, k.transpose(-1, -2)).mul_(scale).reshape(B, nkv, nq // nkv, n, -1)
    pos = (lens - count)[:, None] + i
    key = torch.arange(k.shape[2], device=q.device)
    see = (key <= pos[..., None]) & (key < lens[:, None, None])
    if s["window"]:
        see &= key > pos[..., None] - s["window"]
    sc.masked_fill_(~see[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((key < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p.reshape(B, nkv, -1, p.shape[-1]), v).reshape(B, nkv, nq // nkv, n, D)
    o = (o / total.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(B, n, nq * D)
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(start, t, right=True) - 1
    return o[b, t - start[b]].to(q.dtype)


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)


def _rotated(x, weight, s):
    """Rotation as a complex product: [T][heads][D] in 64 bits."""
    x = x.double().clone()
    if weight is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()
    turn = torch.view_as_complex(s["table"].double()[s["positions"].long()])[:, None]
    rot = s["rot"]
    first = torch.arange(0, rot, 2) if s["interleaved"] else torch.arange(0, rot // 2)
    second = first + (1 if s["interleaved"] else rot // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_rope(s):
    T, nq, nk, D = s["tokens"], s["nq"], s["nk"], s["D"]
    x = s["x"].reshape(T, nq + nk, D)
    q, k = _rotated(x[:, :nq], s["q_weight"], s), _rotated(x[:, nq:], s["k_weight"], s)
    return torch.cat([q, k], 1).reshape(T, -1)


def _stood_for(x):
    """The values that a 4-bit row of x (64 bits) stands for."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    big = torch.maximum(g.amax(-1), -g.amin(-1))
    d = torch.where(g.amax(-1) == big, big, -big).div(-8).half().double()[..., None]
    n = torch.where(d == 0, torch.full_like(g, 8.0), torch.floor(g / d + 8.5)).clamp(0, 15)
    return ((n - 8) * d).reshape(x.shape)


def _exact_append(s):
    T, nq, nkv, D = s["qkv"].shape[0], s["nq"], s["nkv"], s["D"]
    h = s["qkv"].reshape(T, nq + 2 * nkv, D)
    q = _rotated(h[:, :nq], s["q_weight"], s)
    k = _stood_for(_rotated(h[:, nq:nq + nkv], s["k_weight"], s))
    return {"q": q.reshape(T, -1), "k": k.reshape(T, -1), "v": _stood_for(h[:, nq + nkv:].double()).reshape(T, -1)}


def _exact_attn(s):
    nq, nkv, D, w = s["nq"], s["nkv"], s["D"], s["window"]
    lens, new = _lens(s)
    cache, page, dev = s["cache"], s["page"], s["q"].device
    flat = cache.reshape(cache.shape[0], nkv, -1)
    out, at = [], 0
    ch = torch.arange(D, device=dev)
    pl, Gp = _planes(D)
    for b, (L, n) in enumerate(zip(lens, new)):
        tok = torch.arange(L, device=dev)
        pg = s["page_table"][b].long()[tok // page]
        u, t = (tok % page // 16 * 18 * D)[:, None], (tok % 16)[:, None]
        word_k = ((ch // 32 // Gp * 16 + (t >> 1 & 1) * 8 + (t >> 2) * 2 + (t & 1)) * 4 + ch % 32 // 8) * Gp + ch // 32 % Gp
        word_v = (((ch // 32 // Gp * 2 + (t >> 1 & 1)) * 8 + ch % 32 // 4) * 4 + (t >> 2)) * Gp + ch // 32 % Gp
        nib_k, nib_v = ch % 8 + 0 * t, 4 * (t & 1) + ch % 4
        rows = []
        pos = torch.arange(L - n, L, device=dev)[:, None]
        see = tok <= pos
        if w:
            see &= tok > pos - w
        x = s["q"][at:at + n].double().reshape(n, nkv, nq // nkv, D)
        at += n
        for h in range(nkv):
            kv = []
            for word, nib, base in ((word_k, nib_k, 0), (word_v, nib_v, 8 * D)):
                byte = flat[pg[:, None], h, u + base + 4 * word + nib // 2].int()
                val = (byte >> 4 * (nib % 2) & 15) - 8
                so = u + 16 * D + base // 8 + 2 * (t * (D // 32) + ch // 32)
                bits = flat[pg[:, None], h, so].int() + 256 * flat[pg[:, None], h, so + 1].int()
                kv.append(val.double() * bits.to(torch.int16).view(torch.float16).double())
            z = torch.einsum("irc,tc->irt", x[:, h], kv[0]) / math.sqrt(D)
            z = z.masked_fill(~see[:, None], -math.inf)
            rows.append(torch.softmax(z, -1) @ kv[1])
        out.append(torch.stack(rows, 1).reshape(n, nq * D))
    return torch.cat(out)
