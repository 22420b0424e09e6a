"""Cases that time the operators around a quantized cache, adapters and scoring.

A server that answers many users with one quantized model writes keys and
values as codes (``write``: norms, rotation and quantising append, then the rows
read back as the numbers that they stand for), attends over those codes
(``attn``), adds each user's low-rank adapter to the shared projections
(``lora``), and reports log probabilities (``logprobs``). ``run`` computes each
in plain torch operations, or with ``own`` set through the library's entry
points; ``exact`` gives the definitions' values in 64 bits.

Sizes come from the decoder layer of ``qmm_inputs.workloads``: hidden size 5120,
q of 6144 columns, k and v of 1024 (24 query and 4 key heads of 256, or 48 and 8
of 128), gate and up of 17408.
"""
import math

import torch

own = False  # set from outside: False = plain torch operations, True = the library

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
MOST = 65280.0  # values further out are stored as this one


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # One new token into an 8-bit cache: latency.
        dict(name="write_one_token", op="write", M=1, Hq=24, Hkv=4, D=256, R=64, page=16, inter=False, din="f32",
             dtype="bf16", far=262143, bits=8, G=64),
        # A prompt into a 4-bit cache.
        dict(name="write_prompt", op="write", M=8192, Hq=48, Hkv=8, D=128, R=128, page=64, inter=True, din="f32",
             dtype="f16", far=131072, bits=4, G=32),
        # One user, one new token, a short conversation: latency.
        dict(name="attn_one_token", op="attn", B=1, rows=1, ctx=777, Hq=24, Hkv=4, D=256, page=16, window=0, sinks=0,
             dtype="bf16", bits=8, G=64),
        # A full serving batch, one new token each, conversations of 4k to 8k tokens.
        dict(name="attn_batch_decode", op="attn", B=64, rows=1, ctx=8192, Hq=48, Hkv=8, D=128, page=16, window=0,
             sinks=0, dtype="bf16", bits=8, G=64),
        # Speculative verification: up to 8 drafted rows for each of 8 sequences, 4-bit cache.
        dict(name="attn_verify_rows", op="attn", B=8, rows=8, ctx=5000, Hq=24, Hkv=4, D=256, page=64, window=0, sinks=0,
             dtype="f16", bits=4, G=32),
        # One very long context, which is what a 4-bit cache is for.
        dict(name="attn_long_context", op="attn", B=1, rows=4, ctx=131071, Hq=24, Hkv=4, D=256, page=32, window=0,
             sinks=0, dtype="bf16", bits=4, G=64),
        # One user's adapter beside the up projection: latency.
        dict(name="lora_one_row", op="lora", M=1, K=5120, N="17408", n=8, r=16, run=1, dtype="f16"),
        # A serving batch, nearly every row with an adapter of its own, beside the fused q, k and v projections.
        dict(name="lora_batch_qkv", op="lora", M=64, K=5120, N="6144,1024,1024", n=48, r=16, run=1, dtype="bf16"),
        # Prompts of a few users together: long runs of rows with one adapter.
        dict(name="lora_prompts", op="lora", M=2048, K=5120, N="17408", n=4, r=32, run=511, dtype="f16"),
        # One row with its 20 best alternatives: latency.
        dict(name="logprobs_one_row", op="logprobs", M=1, V=131072, n=20, spread=3.0, dtype="f32"),
        # A batch with 5 alternatives.
        dict(name="logprobs_batch", op="logprobs", M=256, V=131072, n=5, spread=2.5, dtype="bf16"),
        # Scoring a prompt's tokens, no alternatives.
        dict(name="logprobs_prompt", op="logprobs", M=1021, V=151001, n=0, spread=3.0, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "attn", "attn", "lora", "logprobs"])
    if op in ("write", "attn"):
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 6, 7, 8, 12])
        page = rng.choice([1, 8, 16, 17, 32, 64, 100, 128, 256])
        c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=rng.choice(["f16", "bf16"]), bits=rng.choice([4, 8]),
                 G=rng.choice([g for g in (32, 64, 128) if g <= D]))
        if op == "write":
            most = min(8192, 8192 * 64 * 128 // ((Hq + 2 * Hkv) * D))  # stays under the largest listed case
            return dict(c, M=_log(rng, 1, most), R=rng.choice([16, D // 4, D // 2, D]), inter=rng.random() < 0.5,
                        din=rng.choice(["f32", "f32", "f16", "bf16"]), far=_log(rng, 1, 262143))
        B = _log(rng, 1, 64)
        rows = rng.choice([1, 1, _log(rng, 1, 16)])
        most = min(131072, 64 * 6000 * 8 * 128 // (B * Hkv * D))
        window = rng.choice([0, 0, _log(rng, 1, 5000)])
        return dict(c, B=B, rows=rows, ctx=max(rows, _log(rng, 1, most)), window=window,
                    sinks=rng.choice([0, 1, 4, 16]) if window else 0)
    if op == "lora":
        K = 32 * _log(rng, 4, 544)
        N = ",".join(str(_log(rng, 40, 17408)) for _ in range(rng.choice([1, 1, 2, 3])))
        r, M = rng.choice([8, 16, 24, 32, 64]), _log(rng, 1, 1024)
        return dict(op=op, M=M, K=K, N=N, n=_log(rng, 1, 48), r=r, run=rng.choice([1, 1, _log(rng, 1, M)]),
                    dtype=rng.choice(["f16", "bf16"]))
    return dict(op=op, M=_log(rng, 1, 512), V=_log(rng, 1000, 160000), n=rng.choice([0, 1, 5, 20, _log(rng, 1, 64)]),
                spread=round(rng.uniform(1.0, 6.0), 2), dtype=rng.choice(["f32", "f16", "bf16"]))


def _lengths(c):
    """Rows and context length of each sequence: ragged, and the same for every seed."""
    B, R, ctx = c["B"], c["rows"], c["ctx"]
    rows = [1 + (R - 1 + 5 * b) % R for b in range(B)]
    lens = [max(rows[b], ctx - (((b * 2654435761) % (1 << 32)) * (ctx // 2) >> 32)) for b in range(B)]
    return rows, lens


def _adapters(c):
    """The adapter of each row, the same for every seed: runs of `run` rows, every eleventh run without one."""
    ids = []
    for i in range(c["M"]):
        k = i // c["run"]
        ids.append(-1 if k % 11 == 10 else (k * 7 + k // 5) % c["n"])
    return ids


def work(case):
    c = case
    if c["op"] == "attn":
        rows, lens = _lengths(c)
        W, S, seen, pairs = c["window"], c["sinks"], 0, 0
        for L, n in zip(lens, rows):
            low = max(0, L - n - W + 1) if W else 0
            seen += L - low + min(S, low)
            for p in range(L - n, L):
                pairs += min(p + 1, W) + max(0, min(S, p + 1 - W)) if W else p + 1
        T = sum(rows)
        row = c["D"] * c["bits"] // 8 + 4 * c["D"] // c["G"]
        return {"bytes": 2 * c["Hkv"] * row * seen + T * c["Hq"] * (4 * c["D"] + 4), "flops": 4 * c["Hq"] * c["D"] * pairs}
    if c["op"] == "write":
        D, kv = c["D"], 2 * c["Hkv"]
        n = c["M"] * (c["Hq"] + kv) * D
        codes = c["M"] * kv * (D * c["bits"] // 8 + 4 * D // c["G"])
        return {"bytes": n * ((4 if c["din"] == "f32" else 2) + 2) + 2 * codes + 8 * c["M"], "flops": 14 * n}
    if c["op"] == "lora":
        ids = [i for i in _adapters(c) if i >= 0]
        used, N, K, r = len(set(ids)), [int(n) for n in c["N"].split(",")], c["K"], c["r"]
        return {"bytes": 2 * c["M"] * K + sum(2 * used * r * (K + n) + 8 * len(ids) * n for n in N),
                "flops": sum(2 * len(ids) * r * (K + n) for n in N)}
    n = c["M"] * c["V"]
    return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + c["M"] * (16 + 8 * c["n"]), "flops": 8 * n}


# --------------------------------------------------------------------------
# The quantized cache in plain operations
# --------------------------------------------------------------------------
def _next_half(h, up):
    """The fp16 number next to each of h, upwards or downwards."""
    i = h.view(torch.int16)
    grows = (h > 0) if up else (h < 0)  # away from zero
    j = torch.where(grows, i + 1, i - 1)
    j = torch.where(h == 0, torch.full_like(i, 1 if up else -32767), j)
    return j.view(torch.float16)


def _quantised(y, bits, G):
    """Codes, scales and biases (float16 [..., D/G]) of the float32 values y [..., D]."""
    g = y.clamp(-MOST, MOST).unflatten(-1, (-1, G))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    b = lo.half()
    b = torch.where(b.float() > lo, _next_half(b, False), b)
    span = hi.double() - b.double()
    levels = 2 ** bits - 1
    s = (span / levels).float().half()
    s = torch.where(s.double() * levels < span, _next_half(s, True), s)
    c = torch.round((g - b.float()) / torch.where(s > 0, s, 1.0).float()).clamp(0, levels)
    return c.flatten(-2).to(torch.uint8), s[..., 0], b[..., 0]


def _packed(codes, s, b, bits):
    """The int32 words of a cache: the codes' bit stream, and scale | bias << 16."""
    if bits == 4:
        codes = codes[..., 0::2] | codes[..., 1::2] << 4
    sb = torch.stack((s, b), -1).contiguous().view(torch.int32)[..., 0]
    return codes.contiguous().view(torch.int32), sb.contiguous()


def _read(words, sb, bits, G):
    """The float16 numbers that words and their (scale, bias) words stand for."""
    codes = words.contiguous().view(torch.uint8)
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    pair = sb.contiguous().view(torch.float16).unflatten(-1, (-1, 2)).float()
    return (codes.float().unflatten(-1, (-1, G)) * pair[..., 0:1] + pair[..., 1:2]).flatten(-2).half()


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    dt = TYPES[c["dtype"]]
    if c["op"] in ("attn", "write"):
        bits, G, D, Hkv, ps = c["bits"], c["G"], c["D"], c["Hkv"], c["page"]

        def pool(pages):
            # values of a cache in use; a chunk at a time, since they are 16 times their codes
            words = torch.empty((pages, Hkv, ps, D * bits // 32), dtype=torch.int32, device=DEV)
            sb = torch.empty((pages, Hkv, ps, D // G), dtype=torch.int32, device=DEV)
            step = max(1, (1 << 26) // (Hkv * ps * D))
            for i in range(0, pages, step):
                n = min(step, pages - i)
                words[i:i + n], sb[i:i + n] = _packed(*_quantised(normal(n, Hkv, ps, D), bits, G), bits)
            return words, sb
    if c["op"] == "attn":
        rows, lens = _lengths(c)
        need = [-(-L // ps) for L in lens]
        total = sum(need) + 3
        pages = torch.randperm(total, generator=g, device=DEV).to(torch.int32)  # in no order, as a pool gives them
        table = torch.zeros((c["B"], max(need)), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = pages[at:at + n]
            at += n
        starts = [0]
        for n in rows:
            starts.append(starts[-1] + n)
        T = starts[-1]
        return dict(op="attn", q=normal(T, c["Hq"], D, dtype=dt, scale=2.0), k=pool(total), v=pool(total), table=table,
                    lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                    starts=torch.tensor(starts, dtype=torch.int32, device=DEV), max_rows=max(rows),
                    max_context=max(lens), window=c["window"], sinks=c["sinks"], scale=1.0 / math.sqrt(D), bits=bits,
                    G=G, out=torch.empty((T, c["Hq"], D), dtype=dt, device=DEV),
                    lse=torch.empty((T, c["Hq"]), dtype=torch.float32, device=DEV))
    if c["op"] == "write":
        M, din = c["M"], TYPES[c["din"]]
        pages = -(-(M + M // 4) // ps) + 1
        slots = torch.randperm(pages * ps, generator=g, device=DEV)[:M].to(torch.int32)
        slots[5::11] = -1  # padding rows of the batch
        return dict(op="write", q=normal(M, c["Hq"], D, dtype=din, scale=1.5), k=normal(M, Hkv, D, dtype=din, scale=1.5),
                    v=normal(M, Hkv, D, dtype=din), q_weight=1.0 + normal(D, scale=0.2), k_weight=1.0 + normal(D, scale=0.2),
                    positions=torch.randint(0, c["far"] + 1, (M,), generator=g, device=DEV, dtype=torch.int32),
                    inv_freq=(1e6 ** (-torch.arange(0, c["R"], 2, dtype=torch.float64) / c["R"])).float().to(DEV),
                    slots=slots, live=torch.nonzero(slots >= 0).flatten(), inter=c["inter"], eps=1e-6, bits=bits, G=G,
                    kc=pool(pages), vc=pool(pages), out=torch.empty((M, c["Hq"], D), dtype=dt, device=DEV),
                    k_rows=torch.empty((M, Hkv, D), dtype=torch.float16, device=DEV),
                    v_rows=torch.empty((M, Hkv, D), dtype=torch.float16, device=DEV))
    if c["op"] == "lora":
        M, K, n, r = c["M"], c["K"], c["n"], c["r"]
        Ns = [int(x) for x in c["N"].split(",")]
        return dict(op="lora", x=normal(M, K, dtype=dt), ids=torch.tensor(_adapters(c), dtype=torch.int32, device=DEV),
                    pairs=[(normal(n, r, K, dtype=dt, scale=K ** -0.5), normal(n, N, r, dtype=dt, scale=r ** -0.5))
                           for N in Ns],
                    scales=0.5 + torch.rand(n, generator=g, device=DEV), ys=[normal(M, N) for N in Ns])
    M, n = c["M"], c["n"]
    return dict(op="logprobs", logits=normal(M, c["V"], dtype=dt, scale=c["spread"]), n=n,
                tokens=torch.randint(0, c["V"], (M,), generator=g, device=DEV, dtype=torch.int32))


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        import affine_group_quantized_qmm_amd as qmm
        if s["op"] == "attn":
            qmm.qmm_paged_attention_quant(s["q"], *s["k"], *s["v"], s["bits"], s["G"], s["table"], s["lens"], s["starts"],
                                          s["max_rows"], s["max_context"], scale=s["scale"], window=s["window"],
                                          sinks=s["sinks"], out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if s["op"] == "write":
            qmm.qmm_qk_norm_rope_quant(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"],
                                       s["inv_freq"], s["slots"], *s["kc"], *s["vc"], s["bits"], s["G"], eps=s["eps"],
                                       interleaved=s["inter"], out=s["out"])
            qmm.qmm_quant_cache_read(*s["kc"], *s["vc"], s["bits"], s["G"], s["slots"], k_out=s["k_rows"],
                                     v_out=s["v_rows"])
            return {"q": s["out"], "k": s["k_rows"], "v": s["v_rows"]}
        if s["op"] == "lora":
            return qmm.qmm_lora(s["x"], s["pairs"], s["ids"], s["ys"], scales=s["scales"])
        lp, rank, entropy, top, top_lp = qmm.qmm_logprobs(s["logits"], s["tokens"], s["n"])
        return {"logprobs": lp, "ranks": rank, "entropy": entropy, "top": top, "top_logprobs": top_lp}
    return {"attn": _plain_attention, "write": _plain_write, "lora": _plain_lora, "logprobs": _plain_logprobs}[s["op"]](s)


def _plain_attention(s):
    q = s["q"]
    T, Hq, D = q.shape
    _, Hkv, ps, _ = s["k"][0].shape
    B, G, R = s["table"].shape[0], Hq // Hkv, s["max_rows"]
    pages = s["table"].long()
    L = pages.shape[1] * ps

    def gathered(cache):
        x = _read(cache[0][pages], cache[1][pages], s["bits"], s["G"])  # [B, pages, Hkv, ps, D]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()

    k = gathered(s["k"])
    starts, lens = s["starts"].long(), s["lens"].long()
    n = starts[1:] - starts[:-1]
    r = torch.arange(R, device=q.device)
    row = (starts[:-1, None] + r).clamp(max=T - 1)
    qf = q[row].float().reshape(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    score = (qf @ k.transpose(2, 3)) * s["scale"]
    del k
    pos = (lens - n)[:, None] + r  # [B, R]
    j = torch.arange(L, device=q.device)
    see = j <= pos[..., None]
    if s["window"]:
        see &= (j > pos[..., None] - s["window"]) | (j < s["sinks"])
    see = see[:, None, :, None, :].expand(B, Hkv, R, G, L).reshape(B, Hkv, R * G, L)
    score = score.masked_fill(~see, float("-inf"))
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ gathered(s["v"])) / total
    lse = (m + torch.log(total))[..., 0]
    o = o.reshape(B, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(B * R, Hq, D)
    lse = lse.reshape(B, Hkv, R, G).permute(0, 2, 1, 3).reshape(B * R, Hq)
    # rows past a sequence's own go to a spare row at the end
    to = torch.where(r < n[:, None], starts[:-1, None] + r, T).reshape(-1)
    out = torch.empty((T + 1, Hq, D), dtype=q.dtype, device=q.device)
    out[to] = o.to(q.dtype)
    all_lse = torch.empty((T + 1, Hq), dtype=torch.float32, device=q.device)
    all_lse[to] = lse
    return {"out": out[:T], "lse": all_lse[:T]}


def _plain_write(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = cos.shape[-1]
    R = 2 * half

    def normed(x, w):
        x = x.float()
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w

    def turned(x):
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["inter"] else (x[..., :half], x[..., half:R])
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1 if s["inter"] else -2).flatten(-2)
        return torch.cat((y, x[..., R:]), -1)

    bits, G, live = s["bits"], s["G"], s["live"]
    ps = s["kc"][0].shape[2]
    slot = s["slots"][live].long()
    s["out"].copy_(turned(normed(s["q"], s["q_weight"])).to(s["out"].dtype))
    rows = {"q": s["out"], "k": s["k_rows"], "v": s["v_rows"]}
    for name, cache, y in (("k", s["kc"], turned(normed(s["k"], s["k_weight"]))), ("v", s["vc"], s["v"].float())):
        words, sb = _packed(*_quantised(y[live], bits, G), bits)
        cache[0][slot // ps, :, slot % ps] = words
        cache[1][slot // ps, :, slot % ps] = sb
        rows[name].zero_()  # padding rows read as zeros
        rows[name][live] = _read(cache[0][slot // ps, :, slot % ps], cache[1][slot // ps, :, slot % ps], bits, G)
    return rows


def _plain_lora(s):
    x, ids = s["x"].float(), s["ids"]
    n = s["scales"].shape[0]
    # every row with every adapter, and the row's own kept: few adapters, no gathered copies of them
    share = torch.where(ids[:, None] == torch.arange(n, device=x.device), s["scales"], 0.0)  # [M, n]
    for (a, b), y in zip(s["pairs"], s["ys"]):
        h = (x @ a.float().flatten(0, 1).T).unflatten(1, (n, -1)) * share[:, :, None]
        y += h.flatten(1) @ b.float().transpose(1, 2).reshape(-1, b.shape[1])
    return s["ys"]


def _plain_logprobs(s):
    x = s["logits"].float()
    M, V = x.shape
    t = s["tokens"].long()[:, None]
    m = x.amax(-1, keepdim=True)
    z = x - m
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total)
    at = x.gather(1, t)
    j = torch.arange(V, device=x.device)
    before = (x > at) | ((x == at) & (j < t))
    top, order = torch.sort(x, dim=-1, descending=True, stable=True) if s["n"] else (x, j.expand(M, V))
    return {"logprobs": (at - m - lse)[:, 0], "ranks": before.sum(-1).to(torch.int32),
            "entropy": (lse - (e * z).sum(-1, keepdim=True) / total)[:, 0], "top": order[:, :s["n"]].to(torch.int32),
            "top_logprobs": top[:, :s["n"]] - m - lse}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attention, "write": _exact_write, "lora": _exact_lora, "logprobs": _exact_logprobs}[case["op"]](s)


def _values(words, sb, bits, G):
    """Code by code with shifts of the words; the nearest fp16 number of scale * code + bias."""
    per = 32 // bits
    shift = torch.arange(per, device=words.device) * bits
    c = (words.long()[..., None] >> shift & (2 ** bits - 1)).flatten(-2).double()
    w = sb.long()
    scale, bias = ((v & 0xFFFF).to(torch.int32).to(torch.int16).view(torch.float16).double() for v in (w, w >> 16))
    return (c * scale.repeat_interleave(G, -1) + bias.repeat_interleave(G, -1)).half().double()


def _exact_attention(s):
    """Sequence by sequence, row by row of queries, over the tokens that are visible."""
    q = s["q"]
    T, Hq, D = q.shape
    _, Hkv, ps, _ = s["k"][0].shape
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for b, L in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        low = 0 if not s["window"] else max(0, L - (last - first) - s["window"] + 1)
        tok = torch.arange(L, device=q.device)
        tok = tok[(tok >= low) | (tok < s["sinks"])]
        page = s["table"][b].long()[tok // ps]
        k, v = (_values(c[page, :, tok % ps], w[page, :, tok % ps], s["bits"], s["G"]) for c, w in (s["k"], s["v"]))
        for t in range(first, last):
            p = L - (last - t)
            n = int((tok <= p).sum())
            vis = tok[:n]
            on = torch.ones(n, dtype=torch.bool, device=q.device)
            if s["window"]:
                on = (vis > p - s["window"]) | (vis < s["sinks"])
            qq = q[t].double().reshape(Hkv, Hq // Hkv, D)
            z = torch.matmul(qq, k[:n].permute(1, 2, 0).contiguous()) * s["scale"]
            z = torch.where(on, z, -math.inf)
            e = torch.logsumexp(z, -1)
            out[t] = torch.matmul(torch.exp(z - e[..., None]), v[:n].permute(1, 0, 2).contiguous()).reshape(Hq, D)
            lse[t] = e.reshape(Hq)
    return {"out": out, "lse": lse}


def _exact_write(s):
    """The rotation as a product of complex numbers; scales and biases by a search of all fp16 numbers."""
    f = s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(f).expand(len(s["positions"]), -1),
                       s["positions"].double()[:, None] * f)[:, None]
    R = 2 * f.numel()

    def whole(x, w):
        x = x.double()
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        if s["inter"]:
            z = torch.view_as_complex(y[..., :R].reshape(*y.shape[:-1], R // 2, 2).contiguous()) * turn
            head = torch.view_as_real(z).reshape(*y.shape[:-1], R)
        else:
            z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
            head = torch.cat((z.real, z.imag), -1)
        return torch.cat((head, y[..., R:]), -1)

    every = torch.arange(-31743, 31744, device=f.device)  # the finite fp16 numbers in rising order
    every = torch.where(every >= 0, every, -32768 - every).to(torch.int16).view(torch.float16).double().contiguous()
    levels = 2 ** s["bits"] - 1

    def stored(y):
        y = y.clamp(-MOST, MOST)
        y = y.reshape(*y.shape[:-1], -1, s["G"])
        b = every[torch.searchsorted(every, y.amin(-1), right=True) - 1]
        step = every[torch.searchsorted(every, (y.amax(-1) - b) / levels)]
        b, step = b[..., None], step[..., None]
        code = torch.where(step > 0, torch.floor((y - b) / torch.where(step > 0, step, 1.0) + 0.5), 0.0).clamp(0, levels)
        value = (step * code + b).half().double()
        return torch.where((s["slots"] >= 0)[:, None, None], value.flatten(-2), 0.0)

    return {"q": whole(s["q"], s["q_weight"]), "k": stored(whole(s["k"], s["k_weight"])), "v": stored(s["v"].double())}


def _exact_lora(s):
    """Adapter by adapter, over the rows that use it."""
    ys = [y.double() for y in s["ys"]]
    for i in sorted(set(s["ids"].tolist()) - {-1}):
        rows = torch.nonzero(s["ids"] == i).flatten()
        for y, (a, b) in zip(ys, s["pairs"]):
            h = s["x"][rows].double() @ a[i].double().T.contiguous()
            y[rows] += s["scales"][i].double() * (h @ b[i].double().T.contiguous())
    return ys


def _exact_logprobs(s):
    """Some rows at a time; ranks by counting in the whole order."""
    parts = []
    for i in range(0, s["logits"].shape[0], 64):
        x = s["logits"][i:i + 64].double()
        t = s["tokens"][i:i + 64].long()
        logp = torch.log_softmax(x, -1)
        values, order = torch.sort(logp if s["logits"].dtype == torch.float64 else x, dim=-1, descending=True, stable=True)
        p = torch.exp(logp)
        rank = torch.argmax((order == t[:, None]).to(torch.int8), -1)
        best = order[:, :s["n"]]
        parts.append((logp.gather(1, t[:, None])[:, 0], rank.to(torch.int32), -(p * logp).sum(-1), best.to(torch.int32),
                      logp.gather(1, best)))
    return dict(zip(("logprobs", "ranks", "entropy", "top", "top_logprobs"), (torch.cat(p) for p in zip(*parts))))
