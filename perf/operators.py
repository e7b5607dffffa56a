"""Workloads of the operators that stand beside the low-bit products in a
serving step: low-rank adapters of many requests (``lora``), the norms around
a block with its gate and residual (``norm``), and the processing of logits
with its top-1 (``logits``).

``own = False`` computes them with elementary torch operations in 32 bits,
``own = True`` through ``bit_matmul_lowbit_amd.lowbit``.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one request with a small adapter on a 2048 -> 6144 projection: a launch-bound call
        dict(name="lora_one_token", op="lora", m=1, k=2048, n=6144, r=16, slots=8, x="f16", y="f32",
             rows="mixed", ragged=False, pad=0),
        # a full decode batch, eight adapters of rank 64, on the gate+up projection of a 27B-class model
        dict(name="lora_batch8_gate_up", op="lora", m=8, k=5120, n=34816, r=64, slots=16, x="f16", y="f32",
             rows="mixed", ragged=False, pad=0),
        # many requests of mixed ranks in arbitrary order, some without an adapter; y is a slice, of an odd
        # width, of a fused projection's output
        dict(name="lora_ragged_200", op="lora", m=200, k=2176, n=1537, r=40, slots=24, x="bf16", y="f32",
             rows="mixed", ragged=True, pad=511),
        # prefill: a few long prompts, each with its adapter, on lowbit_gemm's BF16 output
        dict(name="lora_prefill_4096", op="lora", m=4096, k=5120, n=17408, r=32, slots=8, x="bf16", y="bf16",
             rows="segments", ragged=False, pad=0),
        # one token between two blocks of a small model: a launch-bound call
        dict(name="norm_one_token", op="norm", m=1, k=2048, y="f32", r="f32", x="f16", post="none", pre="rms",
             gate="none"),
        # a decode batch of a 27B-class model: norms on both sides of the block and a gate per row
        dict(name="norm_batch8_gated", op="norm", m=8, k=5120, y="f32", r="f32", x="f16", post="rms", pre="rms",
             gate="row"),
        # layer norms with biases over an odd width, a gate per channel, an FP16 residual
        dict(name="norm_layer_odd", op="norm", m=777, k=1283, y="bf16", r="f16", x="f16", post="layer",
             pre="layer", gate="channel"),
        # prefill of long prompts with a BF16 residual stream
        dict(name="norm_prefill_16384", op="norm", m=16384, k=5120, y="bf16", r="bf16", x="bf16", post="rms",
             pre="rms", gate="none"),
        # greedy decoding of one chat: penalties on a 152k vocabulary, only the token is wanted
        dict(name="logits_greedy_one", op="logits", b=1, n=151936, y="f32", hist=512, bias=0, mask=False,
             out=False),
        # a decode batch under grammars, with biases and all penalties, the logits going on to a sampler
        dict(name="logits_batch8_grammar", op="logits", b=8, n=151936, y="f32", hist=4096, bias=64, mask=True,
             out=True),
        # many short requests on a small odd vocabulary, BF16 logits
        dict(name="logits_ragged_33", op="logits", b=33, n=32003, y="bf16", hist=1000, bias=17, mask=True,
             out=True),
        # a large batch of long conversations
        dict(name="logits_batch64_long", op="logits", b=64, n=151936, y="f32", hist=32768, bias=300, mask=True,
             out=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the ranges that the listed ones stand for; its rows are cut
    so that it moves no more bytes than the largest listed one of its operator."""
    op = rng.choice(["lora", "norm", "logits"])
    if op == "lora":
        x = rng.choice(["f16", "bf16"])
        c = dict(op=op, m=_log_int(rng, 1, 4096), k=128 * _log_int(rng, 1, 136), n=_log_int(rng, 64, 34816),
                 r=8 * _log_int(rng, 1, 16), slots=_log_int(rng, 1, 64), x=x,
                 y="f32" if x == "f16" else rng.choice(["f32", "bf16"]), rows=rng.choice(["mixed", "segments"]),
                 ragged=rng.random() < 0.5, pad=rng.choice([0, 0, 64, rng.randrange(1, 1000)]))
        rows, cap = "m", 3.0e8
    elif op == "norm":
        c = dict(op=op, m=_log_int(rng, 1, 16384), k=_log_int(rng, 64, 17408), y=rng.choice(["f32", "bf16", "f16"]),
                 r=rng.choice(["f32", "bf16", "f16"]), x=rng.choice(["f16", "bf16"]),
                 post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                 gate=rng.choice(["none", "row", "channel"]))
        if rng.random() < 0.5:
            c["k"] = max(128, c["k"] // 128 * 128)  # half of the widths are those of a low-bit matrix
        rows, cap = "m", 6.7e8
    else:
        c = dict(op=op, b=_log_int(rng, 1, 64), n=_log_int(rng, 1000, 151936), y=rng.choice(["f32", "bf16"]),
                 hist=_log_int(rng, 1, 32768), bias=rng.choice([0, 1, _log_int(rng, 2, 300)]),
                 mask=rng.random() < 0.5, out=rng.random() < 0.6)
        rows, cap = "b", 8.0e7
    while c[rows] > 1 and work(c)["bytes"] > cap:
        c[rows] = max(1, int(c[rows] * 0.8))
    if op == "lora":
        while c["slots"] > 1 and work(c)["bytes"] > cap:
            c["slots"] -= 1
    return c


def _ranks(c):
    """Rank of each slot: full, or a fixed mixture (0 among it) of the slot's number."""
    r = c["r"]
    return [[r, (r + 1) // 2, r - 3, 0][s % 4] if c["ragged"] else r for s in range(c["slots"])]


def work(case):
    c = case
    if c["op"] == "lora":
        ranks = _ranks(c)
        mean = sum(ranks) / len(ranks)
        used = min(c["slots"], c["m"])
        byt = (c["m"] * c["k"] * SIZE[c["x"]] + used * mean * (c["k"] + c["n"]) * SIZE[c["x"]]
               + 2 * c["m"] * c["n"] * SIZE[c["y"]])
        return {"bytes": byt, "flops": 2 * c["m"] * mean * (c["k"] + c["n"])}
    if c["op"] == "norm":
        per = SIZE[c["y"]] + 2 * SIZE[c["r"]] + SIZE[c["x"]] + (4 if c["gate"] == "row" else 0)
        vecs = (c["post"] != "none") + (c["post"] == "layer") + (c["pre"] != "none") + (c["pre"] == "layer")
        vecs += c["gate"] == "channel"
        return {"bytes": c["m"] * c["k"] * per + 4 * vecs * c["k"], "flops": 12 * c["m"] * c["k"]}
    b, n = c["b"], c["n"]
    byt = b * n * SIZE[c["y"]] + b * c["hist"] * 3 + b * c["bias"] * 8
    byt += (b * n / 8 if c["mask"] else 0) + (b * n * 4 if c["out"] else 0)
    return {"bytes": byt, "flops": 4 * b * n}


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    def below(hi, *shape):
        return torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.int64)

    s = {"case": c}
    if c["op"] == "lora":
        m, k, n, r, slots = c["m"], c["k"], c["n"], c["r"], c["slots"]
        dt = DTYPES[c["x"]]
        s["x"] = normal(m, k, dtype=dt)
        s["a"] = normal(slots, r, k, sigma=k ** -0.5, dtype=dt)
        s["b"] = normal(slots, n, r, sigma=0.05, dtype=dt)
        s["ranks"] = torch.tensor(_ranks(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
        s["scales"] = uniform(0.5, 2.0, slots)
        order = torch.randperm(slots, generator=g, device="cuda")
        if c["rows"] == "segments":  # one prompt after another
            cuts = torch.sort(below(m + 1, min(slots, m) - 1)).values
            which = torch.searchsorted(cuts, torch.arange(m, device="cuda"), right=True)
        else:  # arbitrary order; with mixed ranks every eleventh row has no adapter
            which = torch.randperm(m, generator=g, device="cuda") % slots
        ids = order[which].to(torch.int32)
        if c["ragged"]:
            ids[10::11] = -1
        s["ids"] = ids
        s["y"] = normal(m, n + c["pad"], dtype=DTYPES[c["y"]])[:, c["pad"]:]
    elif c["op"] == "norm":
        m, k = c["m"], c["k"]
        s["y"] = (normal(m, k) * uniform(0.2, 5.0, m, 1) + 0.1).to(DTYPES[c["y"]])
        s["r"] = normal(m, k, sigma=3.0, dtype=DTYPES[c["r"]])
        s["gate"] = {"none": None, "row": normal(m, k, sigma=0.5) + 1.0 if c["gate"] == "row" else None,
                     "channel": uniform(0.1, 1.0, k)}[c["gate"]]
        s["scale"] = 0.25
        for side in ("post", "pre"):
            s[side + "_w"] = 1.0 + normal(k, sigma=0.2) if c[side] != "none" else None
            s[side + "_b"] = normal(k, sigma=0.2) if c[side] == "layer" else None
        s["r_out"] = torch.empty(m, k, dtype=DTYPES[c["r"]], device="cuda")
        s["x_out"] = torch.empty(m, k, dtype=DTYPES[c["x"]], device="cuda")
    else:
        b, n, hist = c["b"], c["n"], c["hist"]
        s["y"] = normal(b, n, sigma=3.0, dtype=DTYPES[c["y"]])
        # tokens of text: a few are frequent, most are rare; lengths from half of the buffer to all of it
        s["tokens"] = (uniform(0.0, 1.0, b, hist) ** 4 * n).to(torch.int32).clamp_(0, n - 1)
        s["total_len"] = (hist - below(hist // 2 + 1, b)).to(torch.int32)
        s["prompt_len"] = (s["total_len"] * uniform(0.0, 1.0, b)).to(torch.int32)
        s["repetition"] = uniform(1.0, 1.5, b)
        s["frequency"] = uniform(0.0, 0.5, b)
        s["presence"] = uniform(0.0, 0.5, b)
        nb = c["bias"]
        s["bias_ids"] = s["bias_vals"] = s["bias_len"] = None
        if nb:
            s["bias_ids"] = below(n, b, nb).to(torch.int32)
            s["bias_vals"] = normal(b, nb, sigma=5.0)
            s["bias_len"] = (nb - below(nb // 2 + 1, b)).to(torch.int32)
        s["mask"] = None
        if c["mask"]:
            words = (n + 31) // 32
            # a grammar: half of the rows let a few tokens through, the others most
            few = below(1 << 32, b, words) & below(1 << 32, b, words) & below(1 << 32, b, words)
            many = below(1 << 32, b, words) | below(1 << 32, b, words) | below(1 << 32, b, words)
            bits = torch.where((torch.arange(b, device="cuda") % 2 == 0)[:, None], few, many)
            if b > 4:
                bits[3] = 0  # a request whose grammar has no way on
            s["mask"] = (bits - ((bits >> 31) << 32)).to(torch.int32)
        s["out"] = torch.empty(b, n, dtype=torch.float32, device="cuda") if c["out"] else None
        s["idx"] = torch.empty(b, dtype=torch.int32, device="cuda")
        s["val"] = torch.empty(b, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        return {"lora": _own_lora, "norm": _own_norm, "logits": _own_logits}[s["case"]["op"]](s)
    return {"lora": _plain_lora, "norm": _plain_norm, "logits": _plain_logits}[s["case"]["op"]](s)


def _own_lora(s):
    from bit_matmul_lowbit_amd import lowbit

    if "workspace" not in s:  # a serving program allocates it once
        c = s["case"]
        need = lowbit.lowbit_lora_workspace_bytes(c["m"], c["n"], c["k"], c["r"], c["slots"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return lowbit.lowbit_lora_accumulate(s["x"], s["ids"], s["a"], s["b"], s["y"], ranks=s["ranks"],
                                         scales=s["scales"], workspace=s["workspace"])


def _own_norm(s):
    from bit_matmul_lowbit_amd import lowbit

    c = s["case"]
    return lowbit.lowbit_norm_residual(s["y"], s["r"], post=c["post"], post_w=s["post_w"], post_b=s["post_b"],
                                       gate=s["gate"], scale=s["scale"], pre=c["pre"], pre_w=s["pre_w"],
                                       pre_b=s["pre_b"], eps=EPS, r_out=s["r_out"], x_out=s["x_out"])


def _own_logits(s):
    from bit_matmul_lowbit_amd import lowbit

    if "workspace" not in s:  # a serving program allocates it once
        c = s["case"]
        need = lowbit.lowbit_logits_workspace_bytes(c["n"], c["b"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, idx, val = lowbit.lowbit_logits_process(
        s["y"], tokens=s["tokens"], prompt_len=s["prompt_len"], total_len=s["total_len"],
        repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
        bias_vals=s["bias_vals"], bias_len=s["bias_len"], mask=s["mask"], out=s["out"], idx=s["idx"],
        val=s["val"], workspace=s["workspace"])
    return [idx, val] if out is None else [idx, val, out]


def _plain_lora(s):
    # every adapter's product for every row, then the row's own slot and rank are kept
    slots, n, r = s["b"].shape
    m = s["x"].shape[0]
    v = (s["x"].float() @ s["a"].float().view(slots * r, -1).t()).view(m, slots, r)
    mine = s["ids"][:, None] == torch.arange(slots, device="cuda", dtype=torch.int32)
    keep = mine[:, :, None].expand(m, slots, r)
    if s["ranks"] is not None:
        keep = keep & (torch.arange(r, device="cuda") < s["ranks"][:, None])
    v = torch.where(keep, v * s["scales"][:, None], torch.zeros((), device="cuda"))
    delta = v.reshape(m, slots * r) @ s["b"].float().permute(0, 2, 1).reshape(slots * r, n)
    s["y"].copy_(s["y"].float() + delta)
    return s["y"]


def _plain_one_norm(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * w
    return v if b is None else v + b


def _plain_norm(s):
    c = s["case"]
    u = _plain_one_norm(s["y"].float(), c["post"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        u = u * s["gate"]
    r = s["r"].float() + s["scale"] * u
    x = _plain_one_norm(r, c["pre"], s["pre_w"], s["pre_b"])
    return r.to(s["r"].dtype), x.to(s["x_out"].dtype)


def _plain_logits(s):
    c = s["case"]
    b, n, hist = c["b"], c["n"], c["hist"]
    v = s["y"].float()
    if s["bias_ids"] is not None:
        live = torch.arange(c["bias"], device="cuda") < s["bias_len"][:, None]
        v = v + torch.zeros_like(v).scatter_add_(1, s["bias_ids"].long(), s["bias_vals"] * live)
    at = torch.arange(hist, device="cuda")
    live = at < s["total_len"][:, None]
    answer = live & (at >= s["prompt_len"][:, None])
    tokens = s["tokens"].long()
    zero = torch.zeros(b, n, dtype=torch.int32, device="cuda")
    seen = zero.scatter_add(1, tokens, live.int()) > 0
    count = zero.scatter_add(1, tokens, answer.int()).float()
    p = s["repetition"][:, None]
    v = torch.where(seen, torch.where(v > 0, v / p, v * p), v)
    v = v - s["frequency"][:, None] * count
    v = v - s["presence"][:, None] * (count > 0)
    allowed = torch.ones((), dtype=torch.bool, device="cuda")
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        allowed = bits.reshape(b, -1)[:, :n] > 0
        v = torch.where(allowed, v, torch.full((), -math.inf, device="cuda"))
    val = v.amax(dim=1)
    best = allowed & (v == val[:, None])
    idx = torch.where(best, torch.arange(n, device="cuda"), n).amin(dim=1)
    idx = torch.where(idx == n, -1, idx).to(torch.int32)
    return [idx, val, v] if c["out"] else [idx, val]


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"lora": _exact_lora, "norm": _exact_norm, "logits": _exact_logits}[case["op"]](s)


def _exact_lora(s):
    y = s["y"].double()
    ids = s["ids"].tolist()
    for slot in sorted(set(ids)):
        if slot < 0:
            continue
        rows = torch.tensor([i for i, t in enumerate(ids) if t == slot], device="cuda")
        rank = s["a"].shape[1] if s["ranks"] is None else int(s["ranks"][slot])
        a = s["a"][slot, :rank].double()
        b = s["b"][slot, :, :rank].double()
        low = torch.matmul(s["x"][rows].double(), a.t().contiguous())
        y[rows] += float(s["scales"][slot]) * torch.matmul(low, b.t().contiguous())
    return y


def _exact_norm(s):
    c = s["case"]

    def norm(v, kind, w, b):
        if kind == "rms":
            return v / (v.pow(2).sum(1, keepdim=True) / c["k"] + EPS).sqrt() * w.double()
        if kind == "layer":
            mean = v.sum(1, keepdim=True) / c["k"]
            var = (v - mean).pow(2).sum(1, keepdim=True) / c["k"]
            return (v - mean) / (var + EPS).sqrt() * w.double() + b.double()
        return v

    g = 1.0 if s["gate"] is None else s["gate"].double()
    r = s["r"].double() + s["scale"] * g * norm(s["y"].double(), c["post"], s["post_w"], s["post_b"])
    return r, norm(r, c["pre"], s["pre_w"], s["pre_b"])


def _exact_logits(s):
    c = s["case"]
    n = c["n"]
    rows, vals = [], []
    for i in range(c["b"]):
        v = s["y"][i].double()
        if c["bias"]:
            e = int(s["bias_len"][i])
            v.index_add_(0, s["bias_ids"][i, :e].long(), s["bias_vals"][i, :e].double())
        t0, t1 = int(s["prompt_len"][i]), int(s["total_len"][i])
        prompt = torch.bincount(s["tokens"][i, :t0].long(), minlength=n)
        answer = torch.bincount(s["tokens"][i, t0:t1].long(), minlength=n)
        p = float(s["repetition"][i])
        hit = (prompt + answer) > 0
        v[hit] = torch.maximum(v[hit], torch.zeros_like(v[hit])) / p + torch.clamp(v[hit], max=0.0) * p
        v -= float(s["frequency"][i]) * answer
        v[answer > 0] -= float(s["presence"][i])
        if s["mask"] is not None:
            t = torch.arange(n, device="cuda")
            v[((s["mask"][i].long()[t // 32] >> (t % 32)) & 1) == 0] = -math.inf
        rows.append(v)
        vals.append(v.max())
    return [None, torch.stack(vals), torch.stack(rows)] if c["out"] else [None, torch.stack(vals)]
