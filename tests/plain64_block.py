"""Plain numpy forms of rotary positions, the 4-bit cache, attention over it and
sampling (not a test module), with bounds on how far the kernels may be from
them.  Written from the definitions in include/lowbit.h; they share no code with
the library.  tests/test_plain64_block_pins.py holds them to hand-worked
values.
"""
import numpy as np

from tests.plain64 import HALF_STEP, U, rounding

LIMIT = np.float32(16384.0)


# ---------------------------------------------------------------------------
# rotary positions

def frequencies(rot, theta, scaling="none", factor=1.0, trained=1, beta_fast=32.0, beta_slow=1.0):
    """(radians a position of each pair, gain)"""
    i = np.arange(rot // 2)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        pair = [rot * np.log(trained / (b * 2 * np.pi)) / (2 * np.log(theta)) for b in (beta_fast, beta_slow)]
        lo, hi = max(np.floor(pair[0]), 0), min(np.ceil(pair[1]), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * np.log(factor) + 1.0
    return f, 1.0


def cos_sin(positions, turns, gain):
    """FP32 cosines and sines [m][rot / 2]; the phase is exact (Python's whole
    numbers), its rounding to 53 bits the only one before FP32."""
    phase = [[(int(p) * int(t)) % 2 ** 64 for t in turns] for p in positions]
    angle = np.array([[(v - 2 ** 64 if v >= 2 ** 63 else v) / 2.0 ** 64 for v in row] for row in phase]) * (2 * np.pi)
    angle = angle.reshape(len(positions), len(turns))
    return (gain * np.cos(angle)).astype(np.float32), (gain * np.sin(angle)).astype(np.float32)


def rope(x, positions, turns, interleaved=False, gain=1.0, dtype=np.float64):
    """x [m][heads][d], turned with `dtype` arithmetic (FP32: the kernels' own
    order of roundings)."""
    x = x.astype(dtype)
    rot = 2 * len(turns)
    c, s = (t.astype(dtype)[:, None, :] for t in cos_sin(positions, turns, gain))
    at1, at2 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out = x.copy()
    x1, x2 = x[..., at1], x[..., at2]
    out[..., at1] = x1 * c - x2 * s
    out[..., at2] = x2 * c + x1 * s
    return out


def rope_bound(x, positions, turns, interleaved, gain, out_dtype):
    """Two products and a sum in FP32: three roundings for each of the two terms
    (to first order; the cosines are the same FP32 numbers on both sides), and
    one to the output's type.  FP64's cosine is off by less than 2^-50, which
    can move its FP32 rounding by one step: another 2 U."""
    rot = 2 * len(turns)
    at1, at2 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    size = np.zeros(x.shape)
    a = np.abs(x.astype(np.float64))
    size[..., at1] = size[..., at2] = a[..., at1] + a[..., at2]
    out = rope(x, positions, turns, interleaved, gain)
    err = size * abs(gain) * 5 * U
    return err + rounding(np.abs(out) + err, out_dtype)


# ---------------------------------------------------------------------------
# the cache

V_BYTE = (0, 2, 1, 3)


def quantise(x):
    """FP32 x [..][32] -> codes, a, b, by the steps of the definition."""
    x = np.where(np.isnan(x), np.float32(0), x.astype(np.float32)) + np.float32(0)  # -0 becomes 0
    x = np.clip(x, -LIMIT, LIMIT)
    lo, hi = x.min(-1), x.max(-1)
    a = ((hi - lo) * np.float32(16.0 / 15.0)).astype(np.float16)
    b = (lo - a.astype(np.float32)).astype(np.float16)
    off = x - (a.astype(np.float32) + b.astype(np.float32))[..., None]
    step = (a.astype(np.float64) / 16)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.clip(np.rint(off.astype(np.float64) / step), 0, 15)
    return np.where(step > 0, code, 0).astype(np.uint8), a, b


def dequantise(code, a, b):
    """The FP16 numbers that codes [..][32] stand for (FP64 holds the sum
    exactly; numpy rounds it once)."""
    v = a.astype(np.float64)[..., None] * (1 + code / 16.0) + b.astype(np.float64)[..., None]
    return v.astype(np.float16)


def held(x):
    """x [..][d] as the cache holds it."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    return dequantise(*quantise(g)).reshape(x.shape)


def held_bound(x):
    """How far a held value may be from x: half a step, what FP16 takes from a
    and b (the last code may end below the largest value by a's rounding, and
    a value may leave the first one by b's), and the rounding of the value."""
    g = np.clip(x, -LIMIT, LIMIT).astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    span = (g.max(-1) - g.min(-1)) * 16 / 15
    most = np.abs(g).max(-1) + span
    h = HALF_STEP["float16"]
    bound = span / 32 * (1 + h) + 3 * h * most + 2.0 ** -24
    return np.repeat(bound[..., None], 32, -1).reshape(x.shape)


def page_bytes(heads, d, page):
    return heads * page * d * 5 // 4


def put(pages, heads, d, page, slots, k, v):
    """Writes FP32 k, v [m][heads][d] into pages uint8 [n][page_bytes]."""
    n = pages.shape[0]
    g, size = d // 32, page * d // 2
    for i, slot in enumerate(int(s) for s in slots):
        if not 0 <= slot < n * page:
            continue
        p, t = divmod(slot, page)
        for h in range(heads):
            part = pages[p, h * page * d * 5 // 4:(h + 1) * page * d * 5 // 4]
            for which, x in ((0, k), (1, v)):
                code, a, b = quantise(x[i, h].reshape(g, 32))
                flat = code.reshape(-1)
                byte = flat[0::2] | (flat[1::2] << 4)
                ab = np.stack([a, b], -1).view(np.uint8)  # [g][4]
                if which == 0:
                    part[t * d // 2:(t + 1) * d // 2] = byte
                    part[size + t * g * 4:size + (t + 1) * g * 4] = ab.reshape(-1)
                else:
                    base = size + page * g * 4
                    quad, j = divmod(t, 4)
                    part[base:base + size].reshape(page // 4, d // 2, 4)[quad, :, V_BYTE[j]] = byte
                    q = part[base + size:].view(np.uint16).reshape(page // 4, g, 2, 4)
                    q[quad, :, 0, j] = a.view(np.uint16)
                    q[quad, :, 1, j] = b.view(np.uint16)


def get(pages, heads, d, page, slots):
    """(k, v) FP16 [m][heads][d] as the pages hold them; zeros outside."""
    n = pages.shape[0]
    g, size = d // 32, page * d // 2
    out = np.zeros((2, len(slots), heads, d), np.float16)
    for i, slot in enumerate(int(s) for s in slots):
        if not 0 <= slot < n * page:
            continue
        p, t = divmod(slot, page)
        part = pages[p].reshape(heads, -1)
        kc = part[:, t * d // 2:(t + 1) * d // 2]
        kp = part[:, size + t * g * 4:size + (t + 1) * g * 4].copy().view(np.float16).reshape(heads, g, 2)
        base = size + page * g * 4
        quad, j = divmod(t, 4)
        vc = part[:, base:base + size].reshape(heads, page // 4, d // 2, 4)[:, quad, :, V_BYTE[j]]
        vp = part[:, base + size:].copy().view(np.float16).reshape(heads, page // 4, g, 2, 4)[:, quad, :, :, j]
        for which, c, q in ((0, kc, kp), (1, vc, vp)):
            both = np.stack([c & 15, c >> 4], -1).reshape(heads, g, 32)
            out[which, i] = dequantise(both, q[..., 0], q[..., 1]).reshape(heads, d)
    return out[0], out[1]


# ---------------------------------------------------------------------------
# attention

def attention(q, k, v, last, scale, out_dtype):
    """One sequence: q [nq][hq][d], k and v [n][heads][d] FP16, row j sees tokens
    0..last[j] of those in `there`.  Returns (out, lse, bound of out, bound of
    lse), FP64.

    A score is a sum of d products in FP32 in any order, scaled and reduced by
    the maximum: off by at most (d + 4) U of the sum of its terms' magnitudes.  p is
    then off by that much relative, by 2^-21 of the exponential, and by its
    rounding to FP16: 2^-11 relative, or 2^-25 of the largest where it is small.  Both sums are of the rounded p, so what is common to all p
    cancels: an error e of p_t moves the quotient by e |v_t - out|.  The sums over
    n tokens pass no term through more than n / 32 + 600 additions."""
    nq, hq, d = q.shape
    n, heads, _ = k.shape
    group = hq // heads
    out, lse = np.zeros((nq, hq, d)), np.full((nq, hq), -np.inf)
    bound, lbound = np.zeros((nq, hq, d)), np.zeros((nq, hq))
    q, k, v = (t.astype(np.float64) for t in (q, k, v))
    for j in range(nq):
        m = min(max(int(last[j]) + 1, 0), n)
        if m == 0:
            continue
        for h in range(hq):
            kk, vv = k[:m, h // group], v[:m, h // group]
            s = kk @ q[j, h] * scale
            es = np.abs(kk) @ np.abs(q[j, h]) * abs(scale) * (d + 4) * U + np.abs(s) * 4 * U
            p = np.exp(s - s.max())
            total = p.sum()
            o = p @ vv / total
            e = p * (es + 2.0 ** -21 + 2.0 ** -11) + np.minimum(p, 2.0 ** -25)
            depth = (m / 32 + 600) * U
            out[j, h] = o
            lse[j, h] = s.max() + np.log(total)
            err = (e @ (np.abs(vv) + np.abs(o))) / total * 1.01 + depth * 2 * (p @ np.abs(vv)) / total
            bound[j, h] = err + rounding(np.abs(o) + err, out_dtype)
            lbound[j, h] = e.sum() / total * 1.01 + depth + 2.0 ** -20 + np.abs(lse[j, h]) * 4 * U
    return out, lse, bound, lbound


# ---------------------------------------------------------------------------
# sampling

def sample(y, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (token, prob, how far the nearest decision was from falling the
    other way, relative to the sums)."""
    y = y.astype(np.float64)
    n = len(y)
    temperature, top_p, min_p, u = (np.float64(np.float32(t)) for t in (temperature, top_p, min_p, u))
    if not np.any(y > -np.inf) and not np.isnan(y).any():
        return -1, 0.0, 1.0
    if np.isnan(y).any():
        return int(np.nonzero(np.isnan(y))[0][0]), 1.0, 1.0
    if not temperature >= 2.0 ** -20 or y.max() == np.inf:
        return int(np.argmax(y)), 1.0, 1.0
    order = np.argsort(-y, kind="stable")
    w = np.exp((y[order] - y.max()) / temperature)
    margin = 1.0
    if 0 < top_k < n:
        w[top_k:] = 0.0
    keep = w > 0
    if top_p < 1.0:
        total = w.sum()
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        margin = np.min(np.abs(before - top_p * total)[1:], initial=total) / total
        keep &= before < top_p * total
    if min_p > 0.0:
        least = min(min_p, 1.0)
        margin = min(margin, np.min(np.abs(w - least)[w < 1.0], initial=1.0))
        keep &= w >= least
    keep[0] = True
    w = np.where(keep, w, 0.0)
    by_number = np.zeros(n)
    by_number[order] = w
    sums = np.cumsum(by_number)
    target = (0.0 if not u > 0 else min(u, 1 - 2.0 ** -24)) * sums[-1]
    margin = min(margin, np.min(np.abs(sums - target)) / sums[-1])
    token = int(np.nonzero((sums > target) & (by_number > 0))[0][0])
    return token, by_number[token] / sums[-1], margin
