"""Measured cases of the operators beside the quantised products: expert routing, the experts' feed-forward products over
quantised weights, and low-rank adapters of many requests.

* ``route``: T rows of expert scores (softmax or sigmoid of the logits) -> the top_k experts of each row and their
  weights.  The choice goes by score + bias, inside the best ``top_groups`` of ``n_groups`` neighbouring groups (a
  group counts as the sum of its ``group_top`` largest); the lower index wins a tie.  The weights are the scores
  without the bias, divided by their sum where ``renorm``, times ``scale``.
* ``moe_ffn``: y[t] = sum_j weight[t][j] * W_down[e] (silu(W_gate[e] x[t]) * (W_up[e] x[t])) with e = ids[t][j], the
  weights in GGUF blocks (Q8_0, Q4_K, Q6_K); a negative id adds nothing.
* ``lora``: out[t] = y[t] + scale[a] * B[a] (A[a] x[t]) with a = ids[t], a negative id adds nothing.

Blocks (little endian; a row is a whole number of blocks, and columns past its length are not used):
Q8_0: fp16 d, 32 int8 q; w = d q.  Q4_K: fp16 d, fp16 dmin, 12 bytes of 6-bit scales and minima of 8 sub-blocks of 32,
128 bytes of nibbles; w = d sc q - dmin m.  Q6_K: 128 bytes of low nibbles, 64 bytes of high bit pairs, 16 int8
scales, fp16 d; w = d sc (q - 32).
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = {"q8_0": (32, 34), "q4_k": (256, 144), "q6_k": (256, 210)}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the next token of one sequence, 128 experts: latency only
        dict(name="route_1tok", op="route", tokens=1, experts=128, top_k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="f32"),
        # a prompt chunk of the prefill GEMM's size: sigmoid scores, a bias for balance, 4 of 8 groups
        dict(name="route_512_groups", op="route", tokens=512, experts=256, top_k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32"),
        # a long prompt, 16-bit logits (equal ones are common), all groups
        dict(name="route_16384", op="route", tokens=16384, experts=128, top_k=8, score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="bf16"),
        # the next token of one sequence through 8 of 128 experts of 768 x 2048, fp32 as the GEMVs have it
        dict(name="ffn_1tok", op="moe_ffn", tokens=1, experts=128, top_k=8, K=2048, F=768, N=2048, gate="q4_k",
             down="q6_k", pad=0, dtype="f32"),
        # 16 sequences, Q8_0, an odd width (44 blocks a row) and 6 of 64 experts
        dict(name="ffn_16seq", op="moe_ffn", tokens=16, experts=64, top_k=6, K=2048, F=1408, N=2048, gate="q8_0",
             down="q8_0", pad=0, dtype="bf16"),
        # a full decode batch: every expert is read for a few tokens each, three padded places
        dict(name="ffn_64seq", op="moe_ffn", tokens=64, experts=128, top_k=8, K=2048, F=768, N=2048, gate="q4_k",
             down="q4_k", pad=3, dtype="f32"),
        # a prompt chunk of the prefill GEMM's size in 16 bits: about 30 tokens an expert, some with many more
        dict(name="ffn_512tok", op="moe_ffn", tokens=512, experts=128, top_k=8, K=2048, F=768, N=2048, gate="q4_k",
             down="q6_k", pad=0, dtype="f16"),
        # a long prompt: about 256 tokens an expert
        dict(name="ffn_4096tok", op="moe_ffn", tokens=4096, experts=128, top_k=8, K=2048, F=768, N=2048, gate="q4_k",
             down="q4_k", pad=0, dtype="bf16"),
        # the next token of one request beside a 6144 x 4096 projection, rank 16
        dict(name="lora_1tok", op="lora", tokens=1, requests=1, adapters=8, rank=16, K=4096, N=6144, idle=0,
             dtype="f32", wtype="f16"),
        # 64 requests at their next token, 48 adapters, every eighth request without one
        dict(name="lora_64req", op="lora", tokens=64, requests=64, adapters=48, rank=16, K=4096, N=4096, idle=8,
             dtype="f32", wtype="bf16"),
        # prompt chunks of three requests in the 896-wide model's up projection, odd lengths, a small rank
        dict(name="lora_333tok", op="lora", tokens=333, requests=3, adapters=4, rank=8, K=896, N=4864, idle=0,
             dtype="f16", wtype="f16"),
        # long prompts of seven requests beside a 6144 x 4096 projection, rank 64
        dict(name="lora_4096tok", op="lora", tokens=4096, requests=7, adapters=8, rank=64, K=4096, N=6144, idle=0,
             dtype="bf16", wtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "moe_ffn", "moe_ffn", "lora"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "route":
        experts = rng.choice([8, 60, 64, 128, 160, 256, 384, 512])
        groups = rng.choice([1, 1, 4, 8]) if experts % 8 == 0 and experts >= 64 else 1
        top_k = rng.choice([1, 2, 4, 6, 8, 10])
        return dict(op=op, tokens=_log_int(rng, 1, 8192), experts=experts, top_k=min(top_k, experts),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=max(1, groups // 2), group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=dtype)
    if op == "lora":
        K, N = rng.choice([576, 896, 2048, 4096]), rng.choice([576, 1024, 4096, 4864, 6144])
        tokens = _log_int(rng, 1, 4096)
        requests = _log_int(rng, 1, min(tokens, 64))
        return dict(op=op, tokens=tokens, requests=requests, adapters=_log_int(rng, 1, 64),
                    rank=rng.choice([4, 8, 16, 24, 32, 64]), K=K, N=N, idle=rng.choice([0, 0, 4]), dtype=dtype,
                    wtype=rng.choice(["f16", "bf16", "f32"]))
    experts = rng.choice([8, 16, 60, 64, 128])
    top_k = rng.choice([1, 2, 4, 6, 8])
    K, F = rng.choice([576, 896, 1024, 2048]), rng.choice([256, 288, 512, 768, 1408])
    tokens = _log_int(rng, 1, 4096)
    # at most the weights and the products of the largest listed case (wider types take several products)
    while experts * F * K > 2.1e8:
        experts //= 2
    tokens = max(1, min(tokens, int(3e11 / {"f32": 3, "f16": 2, "bf16": 1}[dtype] / (6.0 * top_k * F * K))))
    return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, K=K, F=F, N=K, gate=rng.choice(["q4_k", "q8_0"]),
                down=rng.choice(["q4_k", "q6_k", "q8_0"]), pad=rng.choice([0, 0, min(tokens - 1, 5)]), dtype=dtype)


def _row_bytes(fmt, n):
    per, size = BLOCK[fmt]
    return -(-n // per) * size


def _segments(case):
    """Tokens of each request: uneven, the same for every seed."""
    T, R = case["tokens"], case["requests"]
    part = [0.4 + (i * 0.6180339887498949) % 1.0 for i in range(R)]
    at = [0]
    for i in range(R):
        at.append(max(at[-1] + 1, min(T - (R - 1 - i), round(T * sum(part[:i + 1]) / sum(part)))))
    return [b - a for a, b in zip(at, at[1:])]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    T = case["tokens"]
    if case["op"] == "route":
        E, k = case["experts"], case["top_k"]
        return dict(bytes=T * E * size + T * k * 8 + (4 * E if case["bias"] else 0), flops=6 * T * E)
    if case["op"] == "lora":
        K, N, r = case["K"], case["N"], case["rank"]
        idle = case["idle"]
        seg = _segments(case)
        live = [n for i, n in enumerate(seg) if not (idle and i % idle == idle - 1)]
        used = min(len(live), case["adapters"])
        wsize = 4 if case["wtype"] == "f32" else 2
        return dict(bytes=sum(live) * K * size + 2 * T * N * size + used * (K + N) * r * wsize + 4 * T,
                    flops=2 * sum(live) * r * (K + N))
    E, k, K, F, N = case["experts"], case["top_k"], case["K"], case["F"], case["N"]
    live = T - case["pad"]
    # experts that T rows of k reach (each expert as likely)
    used = E * (1 - (1 - min(k, E) / E) ** live)
    per = 2 * F * _row_bytes(case["gate"], K) + N * _row_bytes(case["down"], F)
    return dict(bytes=used * per + live * K * size + T * N * size + T * k * 8, flops=2 * live * k * F * (2 * K + N))


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _bytes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


def _fp16_bytes(x):
    return x.half().contiguous().view(torch.uint8).reshape(*x.shape, 2)


def _blocks(g, fmt, rows, n, rms):
    """Random blocks of `rows` rows of n columns whose weights have about the given root mean square."""
    per = -(-n // BLOCK[fmt][0])
    spread = torch.exp(_normal(g, rows, per, scale=0.3))
    if fmt == "q8_0":
        return torch.cat([_fp16_bytes(spread * rms / 73), _bytes(g, rows, per, 32)], -1).reshape(rows, -1)
    if fmt == "q6_k":
        sc = torch.randint(-64, 64, (rows, per, 16), generator=g, device="cuda").to(torch.int8).view(torch.uint8)
        return torch.cat([_bytes(g, rows, per, 192), sc, _fp16_bytes(spread * rms / 690)], -1).reshape(rows, -1)
    d = spread * rms / 215
    dmin = d * 7.5 * torch.exp(_normal(g, rows, per, scale=0.1))
    return torch.cat([_fp16_bytes(d), _fp16_bytes(dmin), _bytes(g, rows, per, 140)], -1).reshape(rows, -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dt, T = DT[case["dtype"]], case["tokens"]
    if case["op"] == "route":
        E = case["experts"]
        s["logits"] = (_normal(g, T, E, scale=1.5) + _normal(g, E, scale=0.5)).to(dt)
        s["bias_t"] = _normal(g, E, scale=0.1) if case["bias"] else None
        return s
    if case["op"] == "lora":
        n, r, K, N = case["adapters"], case["rank"], case["K"], case["N"]
        wt = DT[case["wtype"]]
        s["x"], s["y"] = _normal(g, T, K).to(dt), _normal(g, T, N).to(dt)
        s["A"] = _normal(g, n, r, K, scale=K ** -0.5).to(wt)
        s["B"] = _normal(g, n, N, r, scale=0.5 * r ** -0.5).to(wt)
        s["scales"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        order = torch.randperm(n, generator=g, device="cuda").tolist()
        ids = [order[i % n] if not (case["idle"] and i % case["idle"] == case["idle"] - 1) else -1
               for i in range(case["requests"])]
        s["ids"] = torch.tensor(ids, dtype=torch.int32).repeat_interleave(torch.tensor(_segments(case))).cuda()
        return s
    E, k, K, F, N = case["experts"], case["top_k"], case["K"], case["F"], case["N"]
    s["x"] = (_normal(g, T, K) * torch.exp(_normal(g, K, scale=0.3))).to(dt)
    for name, fmt, rows, cols in (("gate_w", case["gate"], E * F, K), ("up_w", case["gate"], E * F, K),
                                  ("down_w", case["down"], E * N, F)):
        s[name] = _blocks(g, fmt, rows, cols, cols ** -0.5)
    # some experts are chosen more often than others
    logits = _normal(g, T, E) + _normal(g, E, scale=0.4)
    top = torch.topk(logits, k, dim=1)
    s["weights"] = torch.softmax(top.values, 1)
    s["ids"] = top.indices.int()
    if case["pad"]:
        s["ids"][T - case["pad"]:] = -1
    # room of the plain form: the tokens of the fullest expert (expert 0 with the padded places)
    s["room"] = int(torch.bincount(s["ids"].clamp(min=0).flatten(), minlength=E).max())
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"route": _run_route, "moe_ffn": _run_ffn, "lora": _run_lora}[s["op"]](s)


def _run_route(s):
    k = s["top_k"]
    if own:
        from quantised_gguf_weight_gb300 import qk
        ids, weights = qk.moe_route(s["logits"], k, score=s["score"], bias=s["bias_t"], n_groups=s["groups"],
                                    top_groups=s["top_groups"], group_top=s["group_top"], renorm=s["renorm"],
                                    scale=s["scale"])
        return {"ids": ids, "weights": weights}
    # 64 bits: the choice between neighbouring scores is in their last places
    z = s["logits"].double()
    if s["score"] == "softmax":
        z = torch.exp(z - z.amax(1, keepdim=True))
        p = z / z.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    c = p if s["bias_t"] is None else p + s["bias_t"].double()
    if s["groups"] > 1:
        gs = c.unflatten(1, (s["groups"], -1)).sort(dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, best, True)
        c = c.masked_fill(~keep.repeat_interleave(c.shape[1] // s["groups"], 1), -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.int(), "weights": (w * s["scale"]).float()}


def _decoded(fmt, blocks, n):
    """Blocks [rows][bytes] -> weights [rows][n] fp32."""
    rows = blocks.shape[0]
    b = blocks.reshape(rows, -1, BLOCK[fmt][1])
    half = lambda at: b[..., at:at + 2].contiguous().view(torch.float16).float()  # noqa: E731
    if fmt == "q8_0":
        w = half(0) * b[..., 2:].contiguous().view(torch.int8).float()
    elif fmt == "q6_k":
        ql, qh = b[..., :128].reshape(rows, -1, 2, 2, 32), b[..., 128:192].reshape(rows, -1, 2, 1, 32)
        low = torch.cat([ql & 15, ql >> 4], 3)
        high = torch.cat([qh & 3, qh >> 2 & 3, qh >> 4 & 3, qh >> 6], 3)
        q = (low | high << 4).float() - 32
        sc = b[..., 192:208].contiguous().view(torch.int8).float() * half(208)
        w = q.reshape(rows, -1, 16, 16) * sc[..., None]
    else:
        f = b[..., 4:16]
        sc = torch.cat([f[..., 0:4] & 63, (f[..., 8:12] & 15) | (f[..., 0:4] >> 6 << 4)], -1).float() * half(0)
        m = torch.cat([f[..., 4:8] & 63, (f[..., 8:12] >> 4) | (f[..., 4:8] >> 6 << 4)], -1).float() * half(2)
        q = b[..., 16:].reshape(rows, -1, 4, 1, 32)
        q = torch.cat([q & 15, q >> 4], 3).reshape(rows, -1, 8, 32).float()
        w = q * sc[..., None] - m[..., None]
    return w.reshape(rows, -1)[:, :n]


def _run_ffn(s):
    x, ids, E, k = s["x"], s["ids"], s["experts"], s["top_k"]
    K, F, N = s["K"], s["F"], s["N"]
    if own:
        from quantised_gguf_weight_gb300 import qk
        return qk.moe_ffn(x, ids, s["weights"], qk.ExpertWeights(s["gate"], s["gate_w"]),
                          qk.ExpertWeights(s["gate"], s["up_w"]), qk.ExpertWeights(s["down"], s["down_w"]), E, F, N)
    flat = ids.flatten().long()
    live = flat >= 0
    token = torch.arange(flat.numel(), device=x.device) // k
    gate_w, up_w, down_w = (s[n].reshape(E, -1, s[n].shape[1]) for n in ("gate_w", "up_w", "down_w"))
    if flat.numel() < E:
        # few rows: each beside its own copy of its expert's weights
        at, place = torch.arange(flat.numel(), device=x.device), torch.zeros_like(flat)
        gate_w, up_w, down_w = (w[flat.clamp(min=0)] for w in (gate_w, up_w, down_w))
        rows = x.float()[token][:, None]
    else:
        # the rows of each expert side by side, in order, at most `room`; those of no expert in a place of their own
        at = torch.where(live, flat, torch.full_like(flat, E))
        order = at.sort(stable=True).indices
        sorted_at = at[order]
        first = torch.searchsorted(sorted_at, torch.arange(E + 1, device=x.device))
        place = torch.empty_like(flat)
        place[order] = torch.arange(flat.numel(), device=x.device) - first[sorted_at]
        rows = torch.zeros(E + 1, s["room"], K, device=x.device)
        rows[at, place] = x.float()[token]
        rows, at = rows[:E], at.clamp(max=E - 1)
    n = gate_w.shape[0]
    g = torch.bmm(rows, _decoded(s["gate"], gate_w.flatten(0, 1), K).reshape(n, F, K).transpose(1, 2))
    u = torch.bmm(rows, _decoded(s["gate"], up_w.flatten(0, 1), K).reshape(n, F, K).transpose(1, 2))
    h = g / (1 + torch.exp(-g)) * u
    o = torch.bmm(h, _decoded(s["down"], down_w.flatten(0, 1), F).reshape(n, N, F).transpose(1, 2))
    o = o[at, place].reshape(-1, k, N)
    w = torch.where(live.reshape(-1, k), s["weights"], torch.zeros_like(s["weights"]))
    return (o * w[..., None]).sum(1).to(x.dtype)


def _run_lora(s):
    x, y, ids = s["x"], s["y"], s["ids"]
    if own:
        from quantised_gguf_weight_gb300 import qk
        return qk.lora(x, y, s["A"], s["B"], ids, scales=s["scales"])
    n, r = s["adapters"], s["rank"]
    v = x.float() @ s["A"].float().reshape(n * r, -1).t()
    mine = (torch.arange(n, device=x.device) == ids[:, None]).float() * s["scales"]
    v = (v.reshape(-1, n, r) * mine[..., None]).reshape(-1, n * r)
    return (y.float() + v @ s["B"].float().transpose(1, 2).reshape(n * r, -1)).to(y.dtype)


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "moe_ffn": _exact_ffn, "lora": _exact_lora}[case["op"]](s)


def _exact_route(s):
    z, E, k = s["logits"].double(), s["experts"], s["top_k"]
    p = torch.softmax(z, 1) if s["score"] == "softmax" else torch.sigmoid(z)
    c = p + s["bias_t"].double() if s["bias_t"] is not None else p.clone()
    each = E // s["groups"]
    index = torch.arange(E, device=z.device)
    if s["groups"] > 1:
        total = torch.stack([c[:, i:i + each].topk(s["group_top"], 1).values.sum(1) for i in range(0, E, each)], 1)
        # groups that are better than each, or as good and before it
        i = torch.arange(s["groups"], device=z.device)
        better = (total[:, None] > total[..., None]) | ((total[:, None] == total[..., None]) & (i < i[:, None]))
        c = torch.where((better.sum(2) < s["top_groups"])[:, index // each], c, torch.full_like(c, -math.inf))
    ids = []
    for _ in range(k):
        top = c.amax(1, keepdim=True)
        i = torch.where(c == top, index, E).amin(1, keepdim=True)
        ids.append(i)
        c = c.scatter(1, i, -math.inf)
    ids = torch.cat(ids, 1)
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.int(), "weights": w * s["scale"]}


def _exact_weights(fmt, blocks, n):
    """Rows of blocks -> weights [rows][n] in 64 bits, column by column of the block."""
    per, size = BLOCK[fmt]
    b = blocks.reshape(blocks.shape[0], -1, size).int()
    dev = blocks.device
    fp16 = lambda at: (b[..., at] + 256 * b[..., at + 1]).to(torch.int16).view(torch.float16).double()[..., None]  # noqa: E731
    signed = lambda v: torch.where(v > 127, v - 256, v).double()  # noqa: E731
    i = torch.arange(per, device=dev)
    if fmt == "q8_0":
        w = fp16(0) * signed(b[..., 2 + i])
    elif fmt == "q6_k":
        h, t, l = i // 128, i % 128 // 32, i % 32
        low = b[..., 64 * h + l + 32 * (t % 2)] >> 4 * (t // 2) & 15
        high = b[..., 128 + 32 * h + l] >> 2 * t & 3
        w = fp16(208) * signed(b[..., 192 + i // 16]) * (low + 16 * high - 32)
    else:
        j = i // 32
        a, m4 = j % 4, j >= 4
        sc = torch.where(m4, (b[..., 12 + a] & 15) + 16 * (b[..., 4 + a] >> 6), b[..., 4 + a] & 63)
        mn = torch.where(m4, (b[..., 12 + a] >> 4) + 16 * (b[..., 8 + a] >> 6), b[..., 8 + a] & 63)
        q = b[..., 16 + 32 * (j // 2) + i % 32] >> 4 * (j % 2) & 15
        w = fp16(0) * (sc * q) - fp16(2) * mn
    return w.reshape(blocks.shape[0], -1)[:, :n]


def _exact_ffn(s):
    x, E, K, F, N = s["x"].double(), s["experts"], s["K"], s["F"], s["N"]
    y = torch.zeros(x.shape[0], N, dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        g = x[t] @ _exact_weights(s["gate"], s["gate_w"][e * F:(e + 1) * F], K).t()
        u = x[t] @ _exact_weights(s["gate"], s["up_w"][e * F:(e + 1) * F], K).t()
        o = (g * torch.sigmoid(g) * u) @ _exact_weights(s["down"], s["down_w"][e * N:(e + 1) * N], F).t()
        y.index_add_(0, t, o * s["weights"][t, j].double()[:, None])
    return y


def _exact_lora(s):
    out = s["y"].double().clone()
    ids = s["ids"].tolist()
    for a in sorted(set(i for i in ids if i >= 0)):
        t = (s["ids"] == a).nonzero()[:, 0]
        out[t] += s["scales"][a].double() * (s["x"][t].double() @ s["A"][a].double().t() @ s["B"][a].double().t())
    return out
