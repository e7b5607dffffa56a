"""Workloads of what stands between the products of a block and after the last
one: rotary positions (``rope``), a cache held in 4 bits as it is written and
read back (``cache``), attention over that cache (``attn``), and drawing a
token from logits (``sample``).

``own = False`` computes them with elementary torch operations, ``own = True``
through ``bit_matmul_lowbit_amd.lowbit``.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
THETA = 1.0e6
CONTEXT = 262144  # positions are drawn below this
TRAINED = 32768  # the length that scaled rotary frequencies were trained at


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # queries of a decode batch of a 27B-class model as the product left them: a quarter of the head turns
        dict(name="rope_batch8", op="rope", m=8, heads=24, d=256, rot=64, inter=False, scaling="none", x="f32",
             out="f16", pad=2048),
        # prefill of long prompts beyond the trained length, the whole head turns, pairs side by side
        dict(name="rope_prefill_8192", op="rope", m=8192, heads=32, d=128, rot=128, inter=True, scaling="yarn",
             x="bf16", out="bf16", pad=0),
        # one token of a small model: rotated, written to the cache, read back; launch-bound
        dict(name="cache_one_token", op="cache", m=1, hq=16, heads=8, d=128, page=16, rot=128, inter=False, x="f32",
             out="f16", order="mixed"),
        # one token of each of 61 chats of a 27B-class model, in pages of their own
        dict(name="cache_batch61", op="cache", m=61, hq=24, heads=4, d=256, page=64, rot=64, inter=False, x="f32",
             out="f16", order="mixed"),
        # a chunk of a long prompt on its way into the cache
        dict(name="cache_prefill_4096", op="cache", m=4096, hq=32, heads=8, d=128, page=16, rot=128, inter=False,
             x="bf16", out="bf16", order="rows"),
        # a long conversation's cache read back, as for another place that holds 16 bits
        dict(name="cache_read_32768", op="read", m=32768, heads=4, d=256, page=64, out="f16", order="rows"),
        # one chat of a small model: latency
        dict(name="attn_one_4096", op="attn", b=1, ctx=4096, q=1, hq=16, heads=8, d=128, page=16, lens="full",
             x="f16", out="f16"),
        # a decode batch of a 27B-class model, short chats and long ones
        dict(name="attn_batch16_mixed", op="attn", b=16, ctx=32767, q=1, hq=24, heads=4, d=256, page=64,
             lens="mixed", x="f16", out="f16"),
        # the longest context of a 27B-class model
        dict(name="attn_one_262144", op="attn", b=1, ctx=262144, q=1, hq=24, heads=4, d=256, page=64, lens="full",
             x="f16", out="f16"),
        # chunks of three prompts, each over what is in the cache already
        dict(name="attn_chunks_2048", op="attn", b=3, ctx=8192, q=2048, hq=32, heads=8, d=128, page=16, lens="mixed",
             x="bf16", out="bf16"),
        # one chat, a preset (temperature 0.5, top-k 20, top-p 0.85) on a 152k vocabulary
        dict(name="sample_one_preset", op="sample", b=1, n=151936, y="f32", kind="preset"),
        # a batch in which every request has its own settings, open ones among them
        dict(name="sample_batch64_mixed", op="sample", b=64, n=151936, y="f32", kind="mixed"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the ranges that the listed ones stand for, cut so that it
    costs no more than the largest listed one of its operator."""
    op = rng.choice(["rope", "cache", "read", "attn", "attn", "sample"])
    d = rng.choice([64, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 8])
    hq = heads * rng.choice([1, 2, 3, 4, 5, 6, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        d = rng.choice([d, 2 * _log_int(rng, 8, 128)])
        x = rng.choice(["f32", "f16", "bf16"])
        c = dict(op=op, m=_log_int(rng, 1, 8192), heads=_log_int(rng, 1, 40), d=d,
                 rot=rng.choice([d, max(2, d // 4 // 2 * 2), 2 * rng.randint(1, d // 2)]),
                 inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]), x=x,
                 out=rng.choice(["f16", "bf16"]) if x == "f32" else x, pad=rng.choice([0, 0, 128, rng.randrange(1, 500)]))
        rows, cap = "m", 1.34e8
    elif op == "cache":
        x = rng.choice(["f32", "bf16", "f16"])
        c = dict(op=op, m=_log_int(rng, 1, 4096), hq=hq, heads=heads, d=d, page=page, rot=rng.choice([d, d // 4]),
                 inter=rng.random() < 0.5, x=x, out="f16" if x == "f32" else x, order=rng.choice(["rows", "mixed"]))
        rows, cap = "m", 1.2e8
    elif op == "read":
        c = dict(op=op, m=_log_int(rng, 1, 32768), heads=heads, d=d, page=page, out=rng.choice(["f16", "bf16"]),
                 order=rng.choice(["rows", "mixed"]))
        rows, cap = "m", 1.8e8
    elif op == "attn":
        q = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 2048)])
        x = rng.choice(["f16", "bf16"])
        c = dict(op=op, b=_log_int(rng, 1, 64), ctx=max(q, _log_int(rng, 1, 65536)), q=q, hq=hq, heads=heads, d=d,
                 page=page, lens=rng.choice(["full", "mixed"]), x=x, out=x)
        while c["b"] > 1 and (c["b"] * c["ctx"] * heads * d > 2.6e8 or _pairs(c) * hq * d * 4 > 2.2e11):
            c["b"] = max(1, int(c["b"] * 0.8))
        while c["ctx"] > q and _pairs(c) * hq * d * 4 > 2.2e11:
            c["ctx"] = max(q, int(c["ctx"] * 0.8))
        return c
    else:
        c = dict(op=op, b=_log_int(rng, 1, 64), n=_log_int(rng, 100, 151936), y=rng.choice(["f32", "bf16", "f16"]),
                 kind=rng.choice(["preset", "mixed", "open"]))
        rows, cap = "b", 4.0e7
    while c[rows] > 1 and work(c)["bytes"] > cap:
        c[rows] = max(1, int(c[rows] * 0.8))
    return c


def _lengths(c):
    """Tokens in the cache of each sequence, and the queries among them."""
    b, ctx, q = c["b"], c["ctx"], c["q"]
    if c["lens"] == "full":
        return [ctx] * b, [q] * b
    lens = [max(1, ctx // (1, 3, 16, 2, 40, 7)[i % 6] - i) for i in range(b)]
    return lens, [min(n, q if q == 1 else max(1, q - 37 * (i % 3))) for i, n in enumerate(lens)]


def _pairs(c):
    """(query, token) pairs of one query head."""
    return sum(q * n - q * (q - 1) // 2 for n, q in zip(*_lengths(c)))


def work(case):
    c = case
    if c["op"] == "rope":
        per = c["m"] * c["heads"] * c["d"]
        return {"bytes": per * (SIZE[c["x"]] + SIZE[c["out"]]) + 4 * c["m"], "flops": 3 * c["m"] * c["heads"] * c["rot"]}
    if c["op"] == "cache":
        kv, q = 2 * c["m"] * c["heads"] * c["d"], c["m"] * c["hq"] * c["d"]
        # k, v and q come in, q goes out; the cache is written and read, and the values go out
        byt = (kv + q) * SIZE[c["x"]] + q * SIZE[c["out"]] + 2 * kv * 0.625 + kv * SIZE[c["out"]]
        return {"bytes": byt, "flops": 10 * kv + 3 * q}
    if c["op"] == "read":
        kv = 2 * c["m"] * c["heads"] * c["d"]
        return {"bytes": kv * (0.625 + SIZE[c["out"]]), "flops": 2 * kv}
    if c["op"] == "attn":
        lens, qs = _lengths(c)
        byt = sum(lens) * c["heads"] * c["d"] * 1.25 + sum(qs) * c["hq"] * c["d"] * (SIZE[c["x"]] + SIZE[c["out"]])
        return {"bytes": byt, "flops": 4 * _pairs(c) * c["hq"] * c["d"]}
    return {"bytes": c["b"] * c["n"] * SIZE[c["y"]], "flops": 20 * c["b"] * c["n"]}


# ---------------------------------------------------------------------------
# the cache: pages of `page` tokens, in each for every head
#   K codes   [page][d / 2]           two values a byte, the even one low
#   K params  [page][d / 32]{a, b}    FP16
#   V codes   [page / 4][d / 2][4]    tokens 0, 1, 2, 3 of four in bytes 0, 2, 1, 3
#   V params  [page / 4][d / 32]{a of 4 tokens, b of 4 tokens}
# A value is FP16(a * (1 + code / 16) + b).

BYTE = (0, 2, 1, 3)


def _page_bytes(c):
    return c["heads"] * c["page"] * c["d"] * 5 // 4


def _views(pages, heads, d, page):
    """K codes, K params, V codes and V params of all pages."""
    g, n = d // 32, pages.shape[0]
    size = page * d // 2
    by_head = pages.view(n, heads, -1)
    kc, kp, vc, vp = by_head.split([size, page * g * 4, size, page * g * 4], dim=2)
    return (kc.unflatten(2, (page, d // 2)), kp.view(torch.float16).unflatten(2, (page, g, 2)),
            vc.unflatten(2, (page // 4, d // 2, 4)), vp.view(torch.float16).unflatten(2, (page // 4, g, 2, 4)))


def _quantise(x, exactly=True):
    """FP32 x [..][d] -> codes [..][d / 32][32], a and b FP16 [..][d / 32]."""
    x = x.unflatten(-1, (-1, 32))
    lo, hi = x.amin(-1), x.amax(-1)
    a = ((hi - lo) * (16.0 / 15.0)).half()
    b = (lo - a.float()).half()
    off = x - (a.float() + b.float())[..., None]
    step = (a.float() / 16.0)[..., None]
    if exactly:  # a quotient next to half a step
        off, step = off.double(), step.double()
    code = torch.where(step > 0, (off / step).round().clamp(0, 15), torch.zeros((), device="cuda", dtype=off.dtype))
    return code.to(torch.uint8), a, b


def _put(pages, c, slots, k, v, exactly=True):
    """Writes FP32 k and v [m][heads][d] at `slots`."""
    kc, kp, vc, vp = _views(pages, c["heads"], c["d"], c["page"])
    at, t = slots.long() // c["page"], slots.long() % c["page"]
    byte = torch.tensor(BYTE, device="cuda")[t % 4]
    for_k, ka, kb = _quantise(k, exactly)
    flat = for_k.flatten(2)
    kc[at, :, t] = flat[..., 0::2] | (flat[..., 1::2] << 4)
    kp[at, :, t] = torch.stack([ka, kb], -1)
    for_v, va, vb = _quantise(v, exactly)
    flat = for_v.flatten(2)
    vc[at, :, t // 4, :, byte] = flat[..., 0::2] | (flat[..., 1::2] << 4)
    vp[at, :, t // 4, :, :, t % 4] = torch.stack([va, vb], -1)


def _get(pages, c, slots, dtype=torch.float32):
    """k and v [..][heads][d] at `slots`, as the values that the cache stands for."""
    kc, kp, vc, vp = _views(pages, c["heads"], c["d"], c["page"])
    at, t = slots.long() // c["page"], slots.long() % c["page"]
    byte = torch.tensor(BYTE, device="cuda")[t % 4]

    def values(codes, a, b):
        both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, 32))
        v = a.to(dtype)[..., None] * (1 + both.to(dtype) / 16) + b.to(dtype)[..., None]
        return v.half().flatten(-2)

    kk, vv = kp[at, :, t], vp[at, :, t // 4, :, :, t % 4]
    return values(kc[at, :, t], kk[..., 0], kk[..., 1]), values(vc[at, :, t // 4, :, byte], vv[..., 0], vv[..., 1])


# ---------------------------------------------------------------------------
# inputs

def _frequencies(rot, scaling):
    """Radians a position of each pair, and what the rotated values are multiplied by."""
    f = [THETA ** (-2.0 * i / rot) for i in range(rot // 2)]
    factor = CONTEXT / TRAINED
    if scaling == "linear":
        return [v / factor for v in f], 1.0
    if scaling == "yarn":  # fast pairs as they are, slow ones by position interpolation, a ramp between
        def pair(turns):
            return rot * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(THETA))

        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        mix = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        return [v / factor * m + v * (1 - m) for v, m in zip(f, mix)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _turns(freqs):
    """Frequencies as 64-bit fractions of a turn."""
    at = [int(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in freqs]
    return torch.tensor([v - 2 ** 64 if v >= 2 ** 63 else v for v in at], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    def keys(*shape):  # keys have channels that stand out, and biases
        x = torch.randn(shape, generator=g, device="cuda")
        x *= torch.where(uniform(0.0, 1.0, *shape[-2:]) < 0.03, 6.0, 1.0)
        return x.add_(normal(*shape[-2:], sigma=0.5))

    def slots_of(tokens, page, order):
        """A slot for each token: one page after another, the pages in any order, or single slots."""
        pages = -(-tokens // page) if order == "rows" else max(-(-tokens // page), min(tokens, 4096))
        perm = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(tokens, device="cuda")
        if order == "rows":
            return pages, (perm[at // page] * page + at % page).to(torch.int32)
        inside = torch.randint(0, page, (tokens,), generator=g, device="cuda") if tokens <= pages else at // pages
        return pages, (perm[at % pages] * page + inside).to(torch.int32)

    s = {"case": c}
    if c["op"] in ("rope", "cache"):
        freqs, s["gain"] = _frequencies(c["rot"], c.get("scaling", "none"))
        s["turns"] = _turns(freqs)
        m = c["m"]
        first = int(torch.randint(0, CONTEXT - m, (1,), generator=g, device="cuda"))
        if c.get("order") == "mixed":
            s["positions"] = torch.randint(0, CONTEXT, (m,), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["positions"] = torch.arange(first, first + m, device="cuda", dtype=torch.int32)
    if c["op"] == "rope":
        # a slice of a fused projection's output
        wide = normal(c["m"], c["heads"] * c["d"] + c["pad"], dtype=DTYPES[c["x"]])
        s["x"] = wide[:, : c["heads"] * c["d"]].unflatten(1, (c["heads"], c["d"]))
        s["out"] = torch.empty(c["m"], c["heads"], c["d"], dtype=DTYPES[c["out"]], device="cuda")
    elif c["op"] == "cache":
        m, hq, h, d = c["m"], c["hq"], c["heads"], c["d"]
        fused = torch.cat([normal(m, hq, d), keys(m, h, d), normal(m, h, d, sigma=0.7)], dim=1).to(DTYPES[c["x"]])
        s["q"], s["k"], s["v"] = fused[:, :hq], fused[:, hq:hq + h], fused[:, hq + h:]
        n, s["slots"] = slots_of(m, c["page"], c["order"])
        s["pages"] = torch.zeros(n, _page_bytes(c), dtype=torch.uint8, device="cuda")
        s["q_out"] = torch.empty(m, hq, d, dtype=DTYPES[c["out"]], device="cuda")
        s["k_out"] = torch.empty(m, h, d, dtype=DTYPES[c["out"]], device="cuda")
        s["v_out"] = torch.empty(m, h, d, dtype=DTYPES[c["out"]], device="cuda")
    elif c["op"] == "read":
        m, h, d = c["m"], c["heads"], c["d"]
        n, s["slots"] = slots_of(m, c["page"], c["order"])
        s["pages"] = torch.zeros(n, _page_bytes(c), dtype=torch.uint8, device="cuda")
        _put(s["pages"], c, s["slots"], keys(m, h, d), normal(m, h, d, sigma=0.7), False)
        s["k_out"] = torch.empty(m, h, d, dtype=DTYPES[c["out"]], device="cuda")
        s["v_out"] = torch.empty(m, h, d, dtype=DTYPES[c["out"]], device="cuda")
    elif c["op"] == "attn":
        lens, qs = _lengths(c)
        h, d, page = c["heads"], c["d"], c["page"]
        need = [-(-n // page) for n in lens]
        perm = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
        s["pages"] = torch.zeros(sum(need), _page_bytes(c), dtype=torch.uint8, device="cuda")
        s["table"] = torch.full((c["b"], max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            s["table"][i, :n] = perm[at:at + n]
            at += n
        every = sum(need) * page
        for start in range(0, every, 65536):
            slots = torch.arange(start, min(every, start + 65536), device="cuda")
            _put(s["pages"], c, slots, keys(slots.numel(), h, d), normal(slots.numel(), h, d, sigma=0.7), False)
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [0]
        for n in qs:
            starts.append(starts[-1] + n)
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda") if c["q"] > 1 else None
        # as sharp as trained heads are: scores of a standard deviation of one to two
        s["q"] = normal(starts[-1], c["hq"], d, dtype=DTYPES[c["x"]])
        s["scale"] = d ** -0.5
        s["out"] = torch.empty(starts[-1], c["hq"], d, dtype=DTYPES[c["out"]], device="cuda")
        s["seq"] = torch.tensor([i for i, n in enumerate(qs) for _ in range(n)], device="cuda")
        s["last"] = torch.tensor([n - q + j for n, q in zip(lens, qs) for j in range(q)], device="cuda")
        s["most_q"] = max(qs)
    else:
        b, n = c["b"], c["n"]
        s["y"] = (normal(b, n, sigma=2.0) + 12.0 * (uniform(0.0, 1.0, b, n) < 3.0 / n)).to(DTYPES[c["y"]])
        s["u"] = uniform(0.0, 1.0, b)

        def mixed(*choices):
            at = torch.randint(0, len(choices), (b,), generator=g, device="cuda")
            return torch.tensor(choices, device="cuda")[at]

        one = torch.ones(b, device="cuda")
        if c["kind"] == "preset":
            s["temperature"], s["top_k"], s["top_p"] = 0.5 * one, (20 * one).to(torch.int32), 0.85 * one
            s["min_p"] = None
        elif c["kind"] == "open":
            s["temperature"], s["top_k"], s["top_p"], s["min_p"] = one, None, None, None
        else:
            s["temperature"] = mixed(0.0, 0.2, 0.5, 0.7, 1.0, 1.3)
            s["top_k"] = mixed(0, 0, 1, 20, 50, 1000, 20000).to(torch.int32)
            s["top_p"] = mixed(0.5, 0.85, 0.95, 1.0, 1.0)
            s["min_p"] = mixed(0.0, 0.0, 0.01, 0.1)
        s["idx"] = torch.empty(b, dtype=torch.int32, device="cuda")
        s["prob"] = torch.empty(b, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        return {"rope": _own_rope, "cache": _own_cache, "read": _own_read, "attn": _own_attn,
                "sample": _own_sample}[s["case"]["op"]](s)
    return {"rope": _plain_rope, "cache": _plain_cache, "read": _plain_read, "attn": _plain_attn,
            "sample": _plain_sample}[s["case"]["op"]](s)


def _own_rope(s):
    from bit_matmul_lowbit_amd import lowbit

    return lowbit.lowbit_rope(s["x"], s["positions"], s["turns"], out=s["out"], interleaved=s["case"]["inter"],
                              gain=s["gain"])


def _own_cache(s):
    from bit_matmul_lowbit_amd import lowbit

    c = s["case"]
    q = lowbit.lowbit_kv_store(s["k"], s["v"], s["slots"], s["pages"], c["page"], positions=s["positions"],
                               turns=s["turns"], interleaved=c["inter"], gain=s["gain"], q=s["q"], q_out=s["q_out"])
    k, v = lowbit.lowbit_kv_load(s["pages"], c["page"], s["slots"], c["heads"], c["d"], k_out=s["k_out"],
                                 v_out=s["v_out"])
    return q, k, v


def _own_read(s):
    from bit_matmul_lowbit_amd import lowbit

    c = s["case"]
    return lowbit.lowbit_kv_load(s["pages"], c["page"], s["slots"], c["heads"], c["d"], k_out=s["k_out"],
                                 v_out=s["v_out"])


def _own_attn(s):
    from bit_matmul_lowbit_amd import lowbit

    c = s["case"]
    if "workspace" not in s:  # a serving program allocates it once
        need = lowbit.lowbit_attention_workspace_bytes(s["q"].shape[0], c["b"], c["hq"], c["heads"], c["d"],
                                                       s["most_q"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return lowbit.lowbit_attention(s["q"], s["pages"], c["page"], s["table"], s["lengths"], q_start=s["q_start"],
                                   max_q=s["most_q"], scale=s["scale"], out=s["out"], workspace=s["workspace"])


def _own_sample(s):
    from bit_matmul_lowbit_amd import lowbit

    if "workspace" not in s:  # a serving program allocates it once
        need = lowbit.lowbit_sample_workspace_bytes(s["case"]["n"], s["case"]["b"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return lowbit.lowbit_sample(s["y"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                min_p=s["min_p"], idx=s["idx"], prob=s["prob"], workspace=s["workspace"])


def _rotate(x, s):
    """FP32 x [m][heads][d]; angles as fractions of a turn, which wrap by themselves."""
    c = s["case"]
    rot = c["rot"]
    half_turns = (s["positions"].long()[:, None] * s["turns"]).double() * 2.0 ** -63
    cos = (torch.cos(math.pi * half_turns) * s["gain"]).float()[:, None]
    sin = (torch.sin(math.pi * half_turns) * s["gain"]).float()[:, None]
    if c["inter"]:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = x[..., : rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    return _rotate(s["x"].float(), s).to(s["out"].dtype)


def _plain_cache(s):
    dtype = s["q_out"].dtype
    _put(s["pages"], s["case"], s["slots"], _rotate(s["k"].float(), s), s["v"].float())
    k, v = _get(s["pages"], s["case"], s["slots"])
    return _rotate(s["q"].float(), s).to(dtype), k.to(dtype), v.to(dtype)


def _plain_read(s):
    k, v = _get(s["pages"], s["case"], s["slots"])
    return k.to(s["k_out"].dtype), v.to(s["v_out"].dtype)


def _plain_attn(s):
    c = s["case"]
    b, heads, page = c["b"], c["heads"], c["page"]
    t = torch.arange(s["table"].shape[1] * page, device="cuda")
    slots = s["table"][:, t // page].clamp(min=0) * page + t % page
    k, v = _get(s["pages"], c, slots)  # [b][tokens][heads][d]
    # every sequence gets as many rows as the one with the most queries
    starts = s["q_start"] if s["q_start"] is not None else torch.arange(b + 1, device="cuda")
    row = torch.arange(s["q"].shape[0], device="cuda") - starts[s["seq"]]
    q = torch.zeros(b, s["most_q"], *s["q"].shape[1:], device="cuda")
    q[s["seq"], row] = s["q"].float()
    last = torch.full((b, s["most_q"]), -1, device="cuda")
    last[s["seq"], row] = s["last"]
    q = q.unflatten(2, (heads, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [b][heads][group * rows][d]
    score = torch.matmul(q, k.float().permute(0, 2, 3, 1).contiguous()) * s["scale"]
    hidden = t > last.repeat(1, c["hq"] // heads)[:, None, :, None]
    score = score.masked_fill(hidden, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3.0e38))
    o = torch.matmul(p, v.float().permute(0, 2, 1, 3).contiguous()) / p.sum(-1, keepdim=True)
    o = o.unflatten(2, (-1, s["most_q"])).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [b][rows][hq][d]
    return o[s["seq"], row].to(s["out"].dtype)


def _plain_sample(s):
    b, n = s["y"].shape
    # as many decimals as keep neighbouring sums of a whole vocabulary apart
    value, token = s["y"].double().sort(dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    w = torch.exp((value - value[:, :1]) / torch.where(greedy, 1.0, t))
    rank = torch.arange(n, device="cuda")
    k = torch.full((b, 1), n, device="cuda") if s["top_k"] is None else s["top_k"].long()[:, None]
    k = torch.where(greedy, 1, torch.where(k <= 0, n, k))
    w = torch.where(rank < k, w, 0.0)
    if s["top_p"] is not None:
        before = w.cumsum(1) - w
        keep = before < s["top_p"].double()[:, None] * w.sum(1, keepdim=True)
        w = torch.where(keep | (rank == 0), w, 0.0)
    if s["min_p"] is not None:
        w = torch.where((w >= s["min_p"].double()[:, None]) | (rank == 0), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, token, w)  # by number again
    total = w.sum(1, keepdim=True)
    over = w.cumsum(1) > s["u"].double()[:, None] * total
    idx = torch.where(over & (w > 0), rank, n).amin(1, keepdim=True)
    prob = w.gather(1, idx.clamp(max=n - 1)) / total
    return idx[:, 0].to(torch.int32), prob[:, 0].float()


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "cache": _exact_cache, "read": _exact_read, "attn": _exact_attn,
            "sample": _exact_sample}[case["op"]](s)


def _turned64(x, s):
    c = s["case"]
    freqs, gain = _frequencies(c["rot"], c.get("scaling", "none"))
    angle = s["positions"].double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full_like(angle, gain), angle)[:, None]
    x = x.double()
    out = x.clone()
    for i in range(c["rot"] // 2):
        p, q = (2 * i, 2 * i + 1) if c["inter"] else (i, i + c["rot"] // 2)
        r = torch.complex(x[..., p], x[..., q]) * z[..., i]
        out[..., p], out[..., q] = r.real, r.imag
    return out


def _exact_rope(s):
    return _turned64(s["x"], s)


def _held64(x):
    """What 4 bits hold of x [m][heads][d], its limits rounded to 16 bits."""
    x = x.double().unflatten(-1, (-1, 32))
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    a = ((hi - lo) * 16 / 15).half().double()
    b = (lo - a).half().double()
    level = torch.arange(16, device="cuda", dtype=torch.float64) / 16
    best = ((x - b) / a.clamp(min=1e-300) - 1).mul(16).round().clamp(0, 15).long()
    return (a * (1 + level[best]) + b).half().double().flatten(-2)


def _exact_cache(s):
    # keys next to half a step may fall to either side of it within 32 bits
    return _turned64(s["q"], s), _held64(_turned64(s["k"], s)), _held64(s["v"])


def _exact_read(s):
    k, v = _get(s["pages"], s["case"], s["slots"], torch.float64)
    return k.double(), v.double()


def _exact_attn(s):
    c = s["case"]
    lens, qs = _lengths(c)
    group, page, out, at = c["hq"] // c["heads"], c["page"], [], 0
    for i, (n, q) in enumerate(zip(lens, qs)):
        t = torch.arange(n, device="cuda")
        k, v = _get(s["pages"], c, s["table"][i].long()[t // page] * page + t % page, torch.float64)
        seen = t[None, :] <= (n - q + torch.arange(q, device="cuda"))[:, None]
        heads = []
        for h in range(c["hq"]):
            kk, vv = k[:, h // group].double(), v[:, h // group].double()
            z = torch.matmul(s["q"][at:at + q, h].double(), kk.t().contiguous()) * s["scale"]
            z = torch.where(seen, z, -math.inf)
            heads.append(torch.matmul(torch.softmax(z, dim=1), vv))
        out.append(torch.stack(heads, 1))
        at += q
    return torch.cat(out)


def _exact_sample(s):
    probs = []
    for i in range(s["case"]["b"]):
        y = s["y"][i].double()
        t = float(s["temperature"][i])
        order = np.argsort(-y.cpu().numpy(), kind="stable")
        k = len(y) if s["top_k"] is None or int(s["top_k"][i]) <= 0 else int(s["top_k"][i])
        order = torch.tensor(order[:1 if t <= 0 else k], device="cuda")
        w = torch.exp((y[order] - y.max()) / (t if t > 0 else 1.0))
        if s["top_p"] is not None:
            share = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), w.cumsum(0)[:-1]]) / w.sum()
            most = max(1, int((share < float(s["top_p"][i])).sum()))
            order, w = order[:most], w[:most]
        if s["min_p"] is not None:
            most = max(1, int((w >= float(s["min_p"][i])).sum()))
            order, w = order[:most], w[:most]
        by_number = order.sort().indices
        sums = w[by_number].cumsum(0)
        pick = min(int((sums <= float(s["u"][i]) * float(sums[-1])).sum()), len(sums) - 1)
        probs.append(w[by_number[pick]] / sums[-1])
    return None, torch.stack(probs)
