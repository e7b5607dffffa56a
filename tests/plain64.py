"""Plain numpy forms, in 64 bits, of the operators beside the low-bit products
(not a test module), with bounds on how far an FP32 kernel may be from them.

They are written from the formulas in include/lowbit.h and share no code with
the library; tests/test_plain64_pins.py holds them to hand-worked values.

U is FP32's unit roundoff: a nearest-even FP32 operation is off by at most U
relative.  A sum in which no term passes through more than d additions is off
by at most d * U * (the sum of the terms' magnitudes), to first order.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
# half the distance between the smallest values: what a rounding to a subnormal is off by
TINY = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


def rounding(v, dtype):
    """How far the nearest value of `dtype` may be from v."""
    return np.abs(v) * HALF_STEP[dtype] + TINY[dtype]


# ---------------------------------------------------------------------------
# norms with gate and residual

def norm(v, kind, w=None, b=None, eps=1e-6):
    if kind in (None, "none"):
        return v
    d = v - v.mean(axis=1, keepdims=True) if kind == "layer" else v
    d = d / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)
    if w is not None:
        d = d * w
    return d if b is None else d + b


def norm_residual(y, r, post=None, post_w=None, post_b=None, gate=None, scale=1.0, pre=None, pre_w=None,
                  pre_b=None, eps=1e-6):
    """(r', x) in 64 bits, x None without pre."""
    if y is not None:
        u = norm(y, post, post_w, post_b, eps)
        r = r + scale * (u if gate is None else u * gate)
    return r, None if pre is None else norm(r, pre, pre_w, pre_b, eps)


def _norm_error(v, ev, kind, w, b, eps):
    """Bound on the error of an FP32 norm of v, itself off by ev.

    A row of k is summed by at least 64 lanes, each adding at most
    k / 64 + 1 of its terms, and joined in at most 16 more additions: d = k /
    64 + 17.  With sigma = sqrt(mean(d^2) + eps) and n = d / sigma:
      mean: off by d U mean|v| + mean(ev); the difference by that, by ev and
        by one rounding;
      sigma^2: off by (d + 3) U relative from its own roundings, and by 2
        sigma sqrt(mean(e^2)) from differences off by e; sigma by half of
        both; the division, the root and the products by 4 U."""
    k = v.shape[1]
    d = k / 64 + 17
    if kind in (None, "none"):
        return ev
    c, e = v, ev
    if kind == "layer":
        mean_abs = np.abs(v).mean(axis=1, keepdims=True)
        c = v - v.mean(axis=1, keepdims=True)
        e = ev + ev.mean(axis=1, keepdims=True) + (d + 1) * U * mean_abs + U * np.abs(c)
    sigma = np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
    n = c / sigma
    rel = (d + 8) * U + np.sqrt((e * e).mean(axis=1, keepdims=True)) / sigma
    out = e / sigma + np.abs(n) * rel
    out = out * (1.0 if w is None else np.abs(w))
    return out + (0.0 if b is None else U * (np.abs(b) + np.abs(n if w is None else n * w)))


def norm_residual_bound(y, r, post, post_w, post_b, gate, scale, pre, pre_w, pre_b, eps, r_dtype, x_dtype):
    """Bounds on the errors of r_out and x_out."""
    zero = np.zeros_like(r)
    er = zero
    rr, x = norm_residual(y, r, post, post_w, post_b, gate, scale, pre, pre_w, pre_b, eps)
    if y is not None:
        u = norm(y, post, post_w, post_b, eps)
        g = 1.0 if gate is None else np.abs(gate)
        er = scale * g * (_norm_error(y, zero, post, post_w, post_b, eps) + 3 * U * np.abs(u)) + U * np.abs(rr)
    ex = None
    if x is not None:
        ex = 1.05 * (_norm_error(rr, er, pre, pre_w, pre_b, eps)) + rounding(x, x_dtype)
    return 1.05 * er + rounding(rr, r_dtype), ex


# ---------------------------------------------------------------------------
# logits

def logits_process(y, tokens=None, prompt_len=None, total_len=None, repetition=None, frequency=None,
                   presence=None, bias_ids=None, bias_vals=None, bias_len=None, mask=None, mask_row=None):
    """(out, idx, val, bound) in 64 bits: a loop over rows and list entries."""
    b, n = y.shape
    out, bound = y.astype(np.float64).copy(), np.zeros((b, n))
    idx, val = np.full(b, -1, np.int64), np.full(b, -np.inf)
    for i in range(b):
        v, e = out[i], bound[i]
        if bias_ids is not None:
            cap = bias_ids.shape[1]
            length = cap if bias_len is None else min(max(int(bias_len[i]), 0), cap)
            add, size = np.zeros(n), np.zeros(n)
            for j in range(length):
                t = int(bias_ids[i, j])
                if 0 <= t < n:
                    add[t] += float(bias_vals[i, j])
                    size[t] += U * abs(add[t])
            with np.errstate(invalid="ignore"):
                v += add
            e += size + U * np.abs(v)
        seen, count = np.zeros(n, bool), np.zeros(n)
        if tokens is not None:
            cap = tokens.shape[1]
            total = cap if total_len is None else min(max(int(total_len[i]), 0), cap)
            prompt = 0 if prompt_len is None else min(max(int(prompt_len[i]), 0), total)
            for j in range(total):
                t = int(tokens[i, j])
                if 0 <= t < n:
                    seen[t] = True
                    count[t] += j >= prompt
        p = 1.0 if repetition is None else float(repetition[i])
        f = 0.0 if frequency is None else float(frequency[i])
        q = 0.0 if presence is None else float(presence[i])
        for t in np.nonzero(seen)[0]:
            factor = 1.0 / p if v[t] > 0 else p
            v[t] *= factor
            e[t] = e[t] * factor + U * abs(v[t])
            if count[t] > 0:
                v[t] -= f * count[t]
                e[t] += U * (f * count[t] + abs(v[t]))
                v[t] -= q
                e[t] += U * abs(v[t])
        allowed = np.ones(n, bool)
        if mask is not None:
            mr = i if mask_row is None else int(mask_row[i])
            if mr >= mask.shape[0]:
                allowed[:] = False
            elif mr >= 0:
                words = mask[mr].astype(np.int64) & 0xFFFFFFFF
                t = np.arange(n)
                allowed = ((words[t // 32] >> (t % 32)) & 1) == 1
        v[~allowed] = -np.inf
        e[~allowed] = 0.0
        if allowed.any():
            w = v[allowed]
            at = int(np.nonzero(np.isnan(w))[0][0]) if np.isnan(w).any() else int(np.argmax(w))
            idx[i], val[i] = np.nonzero(allowed)[0][at], w[at]
    return out, idx, val, bound


# ---------------------------------------------------------------------------
# low-rank adapters

def lora(x, ids, a, b, y, ranks=None, scales=None, y_dtype="float32"):
    """(y', bound).  In the first product no term passes through more than k /
    32 + 128 additions (a chain over k in steps of at least 32 terms, the terms
    of a step, and the joining of the parts of k); in the second through no
    more than r + 16."""
    out = y.astype(np.float64).copy()
    bound = np.zeros_like(out)
    slots, r, k = a.shape
    for i, s in enumerate(int(t) for t in ids):
        if not 0 <= s < slots:
            continue
        rank = r if ranks is None else min(max(int(ranks[s]), 0), r)
        scale = 1.0 if scales is None else float(scales[s])
        aa, bb = a[s, :rank], b[s, :, :rank]
        v = scale * (aa @ x[i])
        ev = abs(scale) * (np.abs(aa) @ np.abs(x[i])) * (k / 32 + 130) * U
        out[i] += bb @ v
        bound[i] = np.abs(bb) @ ev + (np.abs(bb) @ np.abs(v)) * (r + 16) * U + rounding(out[i], y_dtype)
    return out, bound
