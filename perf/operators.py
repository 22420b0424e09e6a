"""Cases that time the attention block's operators and the sampler.

A decode or verify step takes the q, k and v projections through the per-head
norms and the rotation into the paged cache (``qk_norm_rope``), attends over
that cache (``paged_attention``) and, after the last projection, chooses a
token for each row (``sample``). ``run`` computes each of them in plain torch
operations, or with ``own`` set through the library's entry points; ``exact``
gives the definitions' values in 64 bits.

Head layouts come from the decoder layer of ``qmm_inputs.workloads`` (q of
6144 columns, k and v of 1024): 24 query and 4 key heads of 256, or 48 and 8
of 128.
"""
import math

import numpy as np
import torch

own = False  # set from outside: False = plain torch operations, True = the library

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # One user, one new token, a short conversation: latency.
        dict(name="attn_one_token", op="attn", B=1, rows=1, ctx=777, Hq=24, Hkv=4, D=256, page=16, window=0, sinks=0,
             dtype="bf16"),
        # A full serving batch, one new token each, conversations of 4k to 8k tokens.
        dict(name="attn_batch_decode", op="attn", B=64, rows=1, ctx=8192, Hq=48, Hkv=8, D=128, page=16, window=0,
             sinks=0, dtype="bf16"),
        # Speculative verification: up to 8 drafted rows for each of 8 sequences.
        dict(name="attn_verify_rows", op="attn", B=8, rows=8, ctx=5000, Hq=24, Hkv=4, D=256, page=64, window=0, sinks=0,
             dtype="f16"),
        # One very long context: few (sequence, head) pairs, so the length is split.
        dict(name="attn_long_context", op="attn", B=1, rows=4, ctx=131071, Hq=24, Hkv=4, D=256, page=32, window=0,
             sinks=0, dtype="bf16"),
        # A sliding-window layer with four sink tokens in the middle of long generations.
        dict(name="attn_window_sinks", op="attn", B=16, rows=2, ctx=30011, Hq=64, Hkv=8, D=64, page=48, window=2047,
             sinks=4, dtype="f16"),
        # One new token through norms, rotation and cache append: latency.
        dict(name="rope_one_token", op="rope", M=1, Hq=24, Hkv=4, D=256, R=64, page=16, inter=False, din="f32",
             dtype="bf16", far=262143),
        # Verify rows of a batch, some of them padding.
        dict(name="rope_verify_rows", op="rope", M=123, Hq=48, Hkv=8, D=128, R=128, page=16, inter=True, din="f32",
             dtype="f16", far=40000),
        # A prompt.
        dict(name="rope_prompt", op="rope", M=8192, Hq=24, Hkv=4, D=256, R=64, page=64, inter=False, din="f32",
             dtype="bf16", far=131072),
        # One row, unfiltered: latency.
        dict(name="sample_one_plain", op="sample", M=1, V=131072, T=1.0, k=0, p=1.0, minp=0.0, spread=3.0, dtype="f32"),
        # Verify rows with the usual filters.
        dict(name="sample_verify_rows", op="sample", M=16, V=151001, T=0.8, k=50, p=0.9, minp=0.0, spread=3.0,
             dtype="f32"),
        # A batch with a wide nucleus (no top-k).
        dict(name="sample_batch_nucleus", op="sample", M=256, V=131072, T=1.0, k=0, p=0.95, minp=0.0, spread=2.5,
             dtype="bf16"),
        # A small vocabulary with min-p.
        dict(name="sample_small_minp", op="sample", M=32, V=32003, T=1.3, k=1000, p=1.0, minp=0.02, spread=4.0,
             dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "sample"])
    if op == "attn":
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 6, 7, 8, 12])
        B = _log(rng, 1, 64)
        rows = rng.choice([1, 1, _log(rng, 1, 16)])
        most = min(131072, 64 * 6000 * 8 * 128 // (B * Hkv * D))  # stays under the largest listed case
        window = rng.choice([0, 0, _log(rng, 1, 5000)])
        return dict(op=op, B=B, rows=rows, ctx=max(rows, _log(rng, 1, most)), Hq=G * Hkv, Hkv=Hkv, D=D,
                    page=rng.choice([1, 8, 16, 17, 32, 64, 100, 128, 256]), window=window,
                    sinks=rng.choice([0, 1, 4, 16]) if window else 0, dtype=rng.choice(["f16", "bf16"]))
    if op == "rope":
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        M = _log(rng, 1, 8192)
        G = rng.choice([1, 2, 4, 6, 7, 8, 12])
        return dict(op=op, M=M, Hq=G * Hkv, Hkv=Hkv, D=D, R=rng.choice([16, D // 4, D // 2, D]),
                    page=rng.choice([1, 16, 17, 64, 100]), inter=rng.random() < 0.5,
                    din=rng.choice(["f32", "f32", "f16", "bf16"]), dtype=rng.choice(["f16", "bf16"]),
                    far=_log(rng, 1, 262143))
    return dict(op=op, M=_log(rng, 1, 256), V=_log(rng, 1000, 160000), T=round(rng.uniform(0.3, 1.6), 3),
                k=rng.choice([0, 1, _log(rng, 1, 2000)]), p=rng.choice([1.0, round(rng.uniform(0.05, 0.999), 3)]),
                minp=rng.choice([0.0, round(rng.uniform(0.0, 0.3), 4)]), spread=round(rng.uniform(1.0, 6.0), 2),
                dtype=rng.choice(["f32", "f16", "bf16"]))


def _lengths(c):
    """Rows and context length of each sequence: ragged, and the same for every seed."""
    B, R, ctx = c["B"], c["rows"], c["ctx"]
    rows = [1 + (R - 1 + 5 * b) % R for b in range(B)]
    lens = [max(rows[b], ctx - (((b * 2654435761) % (1 << 32)) * (ctx // 2) >> 32)) for b in range(B)]
    return rows, lens


def _visible(c, L, n):
    """Tokens of a sequence that some row sees, and (row, token) pairs."""
    W, S, pairs = c["window"], c["sinks"], 0
    for p in range(L - n, L):
        pairs += p + 1 if W == 0 else min(p + 1, W) + max(0, min(S, p + 1 - W))
    low = 0 if W == 0 else max(0, L - n - W + 1)
    return L - low + min(S, low), pairs


def work(case):
    c = case
    if c["op"] == "attn":
        rows, lens = _lengths(c)
        seen = [_visible(c, L, n) for L, n in zip(lens, rows)]
        T = sum(rows)
        return {"bytes": 4 * c["Hkv"] * c["D"] * sum(s for s, _ in seen) + T * c["Hq"] * (4 * c["D"] + 4),
                "flops": 4 * c["Hq"] * c["D"] * sum(p for _, p in seen)}
    if c["op"] == "rope":
        n = c["M"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": n * ((4 if c["din"] == "f32" else 2) + 2) + 8 * c["M"], "flops": 10 * n}
    n = c["M"] * c["V"]
    return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + 28 * c["M"], "flops": 10 * n}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    dt = TYPES[c["dtype"]]
    if c["op"] == "attn":
        rows, lens = _lengths(c)
        ps = c["page"]
        need = [-(-L // ps) for L in lens]
        total = sum(need) + 3
        pages = torch.randperm(total, generator=g, device=DEV).to(torch.int32)  # pages in no order, as a pool gives them
        table = torch.zeros((c["B"], max(need)), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = pages[at:at + n]
            at += n
        shape = (total, c["Hkv"], ps, c["D"])
        starts = [0]
        for n in rows:
            starts.append(starts[-1] + n)
        T = starts[-1]
        return dict(op="attn", q=normal(T, c["Hq"], c["D"], dtype=dt, scale=2.0), k_cache=normal(*shape, dtype=dt),
                    v_cache=normal(*shape, dtype=dt), table=table,
                    lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                    starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                    max_rows=max(rows), max_context=max(lens), window=c["window"], sinks=c["sinks"],
                    scale=1.0 / math.sqrt(c["D"]),
                    out=torch.empty((T, c["Hq"], c["D"]), dtype=dt, device=DEV),
                    lse=torch.empty((T, c["Hq"]), dtype=torch.float32, device=DEV))
    if c["op"] == "rope":
        M, D, ps = c["M"], c["D"], c["page"]
        din = TYPES[c["din"]]
        pool = -(-(M + M // 4) // ps) + 1
        slots = torch.randperm(pool * ps, generator=g, device=DEV)[:M].to(torch.int32)
        slots[5::11] = -1  # padding rows of the batch
        return dict(op="rope", q=normal(M, c["Hq"], D, dtype=din, scale=1.5), k=normal(M, c["Hkv"], D, dtype=din, scale=1.5),
                    v=normal(M, c["Hkv"], D, dtype=din),
                    q_weight=1.0 + normal(D, scale=0.2), k_weight=1.0 + normal(D, scale=0.2),
                    positions=torch.randint(0, c["far"] + 1, (M,), generator=g, device=DEV, dtype=torch.int32),
                    inv_freq=(1e6 ** (-torch.arange(0, c["R"], 2, dtype=torch.float64) / c["R"])).float().to(DEV),
                    slots=slots, live=torch.nonzero(slots >= 0).flatten(), inter=c["inter"], eps=1e-6,
                    k_cache=normal(pool, c["Hkv"], ps, D, dtype=dt), v_cache=normal(pool, c["Hkv"], ps, D, dtype=dt),
                    out=torch.empty((M, c["Hq"], D), dtype=dt, device=DEV))
    M = c["M"]
    temperature = c["T"] * (0.75 + 0.5 * torch.rand(M, generator=g, device=DEV))
    temperature[7::8] = 0.0  # some users of a batch ask for the largest logit
    return dict(op="sample", logits=normal(M, c["V"], dtype=dt, scale=c["spread"]),
                u=torch.rand(M, generator=g, device=DEV), temperature=temperature,
                top_k=torch.full((M,), c["k"], dtype=torch.int32, device=DEV),
                top_p=torch.full((M,), c["p"], dtype=torch.float32, device=DEV),
                min_p=torch.full((M,), c["minp"], dtype=torch.float32, device=DEV),
                tokens=torch.empty(M, dtype=torch.int32, device=DEV),
                logprobs=torch.empty(M, dtype=torch.float32, device=DEV))


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        import affine_group_quantized_qmm_amd as qmm
        if s["op"] == "attn":
            qmm.qmm_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["starts"],
                                    s["max_rows"], s["max_context"], scale=s["scale"], window=s["window"],
                                    sinks=s["sinks"], out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if s["op"] == "rope":
            qmm.qmm_qk_norm_rope(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"],
                                 s["slots"], s["k_cache"], s["v_cache"], eps=s["eps"], interleaved=s["inter"],
                                 out=s["out"])
            return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        qmm.qmm_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], tokens=s["tokens"],
                       logprobs=s["logprobs"])
        return {"tokens": s["tokens"], "logprobs": s["logprobs"]}
    return {"attn": _plain_attention, "rope": _plain_rope, "sample": _plain_sample}[s["op"]](s)


def _plain_attention(s):
    q, kc = s["q"], s["k_cache"]
    T, Hq, D = q.shape
    _, Hkv, ps, _ = kc.shape
    B, G, R = s["table"].shape[0], Hq // Hkv, s["max_rows"]
    pages = s["table"].long()
    L = pages.shape[1] * ps
    k = kc[pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
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
    v = s["v_cache"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
    o = (p @ v) / total
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


def _plain_rope(s):
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

    dt, ps = s["out"].dtype, s["k_cache"].shape[2]
    live = s["live"]
    slot = s["slots"][live].long()
    s["out"].copy_(turned(normed(s["q"], s["q_weight"])).to(dt))
    s["k_cache"][slot // ps, :, slot % ps] = turned(normed(s["k"], s["k_weight"]))[live].to(dt)
    s["v_cache"][slot // ps, :, slot % ps] = s["v"][live].float().to(dt)
    return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_sample(s):
    # 64 bits: a token next to a border must not depend on the order of the sums
    x, order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    rank = torch.arange(x.shape[-1], device=x.device)
    w = torch.exp((x.double() - x[:, :1].double()) / torch.where(t > 0, t, 1.0))
    w = torch.where((t > 0) | (rank == 0), w, 0.0)
    k = s["top_k"][:, None]
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    cum = torch.cumsum(w, -1)
    p = s["top_p"].double()[:, None]
    w = torch.where(((p >= 1) | (cum - w < p * cum[:, -1:])) & (w >= s["min_p"].double()[:, None]), w, 0.0)
    cum = torch.cumsum(w, -1)
    at = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(-1, keepdim=True)
    return {"tokens": order.gather(1, at)[:, 0].to(torch.int32),
            "logprobs": torch.log(w.gather(1, at) / cum[:, -1:])[:, 0].float()}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attention, "rope": _exact_rope, "sample": _exact_sample}[case["op"]](s)


def _exact_attention(s):
    """Sequence by sequence, row by row of queries, over the tokens that are visible."""
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    T, Hq, D = q.shape
    Hkv, ps = kc.shape[1], kc.shape[2]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for b, L in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        low = 0 if not s["window"] else max(0, L - (last - first) - s["window"] + 1)
        tok = torch.arange(L, device=q.device)
        tok = tok[(tok >= low) | (tok < s["sinks"])]
        page = s["table"][b].long()[tok // ps]
        k, v = kc[page, :, tok % ps].double(), vc[page, :, tok % ps].double()  # [n, Hkv, D]
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


def _exact_rope(s):
    """The rotation as a product of complex numbers."""
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

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    ps = kc.shape[2]
    k = whole(s["k"], s["k_weight"])
    m = torch.nonzero(s["slots"] >= 0).flatten()
    slot = s["slots"][m].long()
    kc[torch.div(slot, ps, rounding_mode="floor"), :, slot.remainder(ps)] = k[m]
    vc[torch.div(slot, ps, rounding_mode="floor"), :, slot.remainder(ps)] = s["v"][m].double()
    return {"q": whole(s["q"], s["q_weight"]), "k_cache": kc, "v_cache": vc}


def _exact_sample(s):
    """Row by row on the host: sort, cut the prefix, search the cumulative sum."""
    x = s["logits"].double().cpu().numpy()
    u, T, p, mp = (s[n].double().cpu().numpy() for n in ("u", "temperature", "top_p", "min_p"))
    k = s["top_k"].cpu().numpy()
    tokens, logprobs = [], []
    for i in range(len(x)):
        order = np.argsort(-x[i], kind="stable")
        if k[i] > 0:
            order = order[:k[i]]
        if T[i] <= 0:
            order = order[:1]
        w = np.exp((x[i][order] - x[i][order[0]]) / (T[i] if T[i] > 0 else 1.0))
        cum = np.cumsum(w)
        n = len(w) if p[i] >= 1 else int(np.searchsorted(np.concatenate(([0.0], cum[:-1])), p[i] * cum[-1], "left"))
        n = max(1, min(n, int((w >= mp[i]).sum())))
        cum = cum[:n]
        at = min(int(np.searchsorted(cum, u[i] * cum[-1], "right")), n - 1)
        tokens.append(int(order[at]))
        logprobs.append(math.log(w[at] / cum[-1]))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "logprobs": torch.tensor(logprobs, dtype=torch.float64)}
