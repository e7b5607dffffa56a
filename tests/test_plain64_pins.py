"""The 64-bit plain forms that the operators beside the products are held to,
against hand-worked values and independent identities (CPU)."""
import numpy as np
import pytest

from tests import plain64


def test_norms_by_hand():
    v = np.array([[3.0, 4.0]])
    # mean square 12.5, eps 0: 3 / sqrt(12.5)
    assert np.allclose(plain64.norm(v, "rms", eps=0.0), [[3 / 12.5 ** 0.5, 4 / 12.5 ** 0.5]], rtol=1e-15)
    # mean 3.5, deviations -+0.5, variance 0.25
    assert np.allclose(plain64.norm(v, "layer", np.array([2.0, 3.0]), np.array([10.0, 20.0]), 0.0), [[8.0, 23.0]])
    assert plain64.norm(v, "none") is v
    # a zero row stays finite through eps; a row of one element has no variance
    assert np.array_equal(plain64.norm(np.zeros((1, 4)), "rms"), np.zeros((1, 4)))
    assert np.array_equal(plain64.norm(np.array([[7.0]]), "layer", np.array([5.0]), np.array([0.25])), [[0.25]])


def test_norm_residual_by_hand():
    y, r = np.array([[1.0, -1.0]]), np.array([[2.0, 4.0]])
    rr, x = plain64.norm_residual(y, r, gate=np.array([3.0, 5.0]), scale=0.5, pre="rms", eps=0.0)
    assert np.array_equal(rr, [[3.5, 1.5]])
    assert np.allclose(x, rr / np.sqrt((3.5 ** 2 + 1.5 ** 2) / 2))
    rr, x = plain64.norm_residual(None, r, pre="layer", eps=0.0)
    assert rr is r and np.allclose(x, [[-1.0, 1.0]])


def test_logits_by_hand():
    y = np.array([[4.0, -4.0, 1.0, 0.0, 8.0, 2.0]])
    out, idx, val, _ = plain64.logits_process(
        y, tokens=np.array([[0, 1, 1, 4, 4, -1, 6, 5]]), prompt_len=[2], total_len=[7],
        repetition=[2.0], frequency=[0.5], presence=[0.25],
        bias_ids=np.array([[2, 2, 5, 99]]), bias_vals=np.array([[1.0, 2.0, 50.0, 50.0]]), bias_len=[2])
    # 0: prompt only, 4 / 2;  1: prompt and once after, -4 * 2 - 0.5 - 0.25;  2: biased by 1 + 2;
    # 4: twice after, 8 / 2 - 1 - 0.25;  5: past the length, its bias too
    assert np.array_equal(out, [[2.0, -8.75, 4.0, 0.0, 2.75, 2.0]])
    assert idx[0] == 2 and val[0] == 4.0
    mask = np.array([[0b101001], [0], [0b111111]], np.int64).astype(np.int32)
    out, idx, val, _ = plain64.logits_process(np.repeat(y, 4, 0), mask=mask, mask_row=[0, 1, -1, 3])
    assert np.array_equal(out[0], [4.0, -np.inf, -np.inf, 0.0, -np.inf, 2.0])
    assert list(idx) == [0, -1, 4, -1] and val[1] == val[3] == -np.inf
    ties = np.array([[1.0, 3.0, 3.0, np.nan], [-np.inf] * 4])
    _, idx, val, _ = plain64.logits_process(ties, mask=np.array([[0b0110], [0b1100]], np.int32))
    assert list(idx) == [1, 2] and list(val) == [3.0, -np.inf]
    assert plain64.logits_process(ties)[1][0] == 3  # NaN is largest


def test_lora_by_hand_and_as_one_matrix():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 1.0], [2.0, 0.0]]])  # one slot, r = 2, k = 2
    b = np.array([[[1.0, 10.0], [0.0, 1.0], [5.0, 5.0]]])  # n = 3
    y = np.ones((3, 3))
    out, bound = plain64.lora(x, [0, -1, 1], a, b, y, scales=[0.5])
    # v = 0.5 * (3, 2): 1.5 + 10, 1, 12.5
    assert np.array_equal(out, [[12.5, 2.0, 13.5], [1, 1, 1], [1, 1, 1]])
    assert (bound[0] > 0).all() and not bound[1:].any()
    out, _ = plain64.lora(x, [0, 0, 0], a, b, y, ranks=[1])
    assert np.array_equal(out, y + np.array([[3.0], [7.0], [11.0]]) * np.array([1.0, 0.0, 5.0]))
    g = np.random.default_rng(3)
    a, b, x = g.standard_normal((4, 8, 16)), g.standard_normal((4, 5, 8)), g.standard_normal((9, 16))
    ids, y = g.integers(0, 4, 9), g.standard_normal((9, 5))
    out, _ = plain64.lora(x, ids, a, b, y)
    want = np.stack([y[i] + (b[s] @ a[s]) @ x[i] for i, s in enumerate(ids)])
    assert np.allclose(out, want, rtol=1e-12)


def _planted(name):
    """A copy of the plain module with one line changed."""
    import types

    changes = {
        "variance about zero": ('v - v.mean(axis=1, keepdims=True) if kind == "layer" else v\n    d = d /',
                                'v\n    d = d /'),
        "gate dropped": ("(u if gate is None else u * gate)", "u"),
        "penalty by division alone": ("1.0 / p if v[t] > 0 else p", "1.0 / p"),
        "prompt counted": ("count[t] += j >= prompt", "count[t] += 1"),
        "presence per repetition": ("v[t] -= q", "v[t] -= q * count[t]"),
        "bias without its length": ("for j in range(length):", "for j in range(cap):"),
        "rank past the slot's": ("min(max(int(ranks[s]), 0), r)", "r"),
        "scale dropped": ("v = scale * (aa @ x[i])", "v = aa @ x[i]"),
    }
    old, new = changes[name]
    source = open(plain64.__file__).read()
    assert source.count(old) == 1, name
    mod = types.ModuleType("planted")
    exec(compile(source.replace(old, new), "planted", "exec"), mod.__dict__)
    return mod


@pytest.mark.parametrize("name", ["variance about zero", "gate dropped", "penalty by division alone",
                                  "prompt counted", "presence per repetition", "bias without its length",
                                  "rank past the slot's", "scale dropped"])
def test_pins_fail_for_a_planted_mistake(name, monkeypatch):
    monkeypatch.setitem(globals(), "plain64", _planted(name))
    failed = 0
    for pin in (test_norms_by_hand, test_norm_residual_by_hand, test_logits_by_hand,
                test_lora_by_hand_and_as_one_matrix):
        try:
            pin()
        except AssertionError:
            failed += 1
    assert failed, name
