"""Pins of the oracle's tree forward (head norms with rotation, tree attention,
tree sampling) against numpy and against worked examples, and planted mistakes
in copies of its source, each of which a pin has to catch."""
import os
import subprocess

import numpy as np
import pytest

import oracle
from speculative_decoding_verification_56_gb300 import synth

SRC = os.path.join(os.path.dirname(oracle.__file__), "spec_oracle.c")


@pytest.fixture(scope="module")
def lib():
    oracle.build()
    return None


def bf16(x):
    return synth.f32_to_bf16_bits(np.asarray(x, np.float32))


def wide(b):
    return synth.bf16_bits_to_f32(b).astype(np.float64)


def softmax(z):
    e = np.exp(z - z.max(axis=-1, keepdims=True))
    return e / e.sum(axis=-1, keepdims=True)


# ---------------------------------------------------------------------------
# tree sampling
# ---------------------------------------------------------------------------

def pin_sample_worked_example(lib):
    # probabilities 0.1, 0.2, 0.3, 0.4: u = 0.25 draws token 1, u = 0.3 token 2
    z = np.log(np.array([0.1, 0.2, 0.3, 0.4], np.float32))
    rows = np.stack([z, z[::-1], z, z])[None].astype(np.float32)
    par, tok = np.array([[-1, 0, 0, 1]], np.int32), np.array([[0, 2, 1, 3]], np.int32)
    o = oracle.verify_tree_sample(rows, tok, par, [[0.25, 0.95, 0.5]], 1.0, 2, dtype="f32", lib=lib)
    # token 1 at the root: node 2 (row 2); u = 0.95 there draws token 3, a leaf's last
    assert o["path_nodes"].tolist() == [[0, 2, -1]] and o["out_tokens"].tolist() == [[1, 3, -1]]
    assert np.allclose(o["out_probs"], [[0.2, 0.4, 0]]) and o["accepted_len"].tolist() == [1]
    assert abs(o["margin"][0] - 0.05) < 1e-6
    o = oracle.verify_tree_sample(rows, tok, par, [[0.55, 0.05, 0.5]], 1.0, 2, dtype="f32", lib=lib)
    # token 2: node 1, whose row is reversed (0.4 first): token 0, which node 3 does not hold
    assert o["path_nodes"].tolist() == [[0, 1, -1]] and o["out_tokens"].tolist() == [[2, 0, -1]]
    # temperature 2 takes square roots
    o = oracle.verify_tree_sample(rows[:, :1], tok[:, :1], par[:, :1], [[0.2]], 2.0, 0, dtype="f32", lib=lib)
    w = np.sqrt([0.1, 0.2, 0.3, 0.4])
    assert np.isclose(o["out_probs"][0, 0], w[o["out_tokens"][0, 0]] / w.sum())


def pin_sample_equals_one_by_one_drawing(lib):
    rng = np.random.default_rng(0)
    B, N, V, depth = 40, 14, 6, 4
    z = rng.standard_normal((B, N, V)).astype(np.float32)
    par = np.stack([synth.make_tree_parents(rng, N, max_depth=depth) for _ in range(B)]).astype(np.int32)
    tok = rng.integers(0, V, (B, N)).astype(np.int32)
    u = rng.random((B, depth + 1)).astype(np.float32)
    o = oracle.verify_tree_sample(z, tok, par, u, 0.75, depth, dtype="f32", lib=lib)
    lengths = set()
    for b in range(B):
        cur, d = 0, 0
        while True:
            c = np.cumsum(softmax(z[b, cur].astype(np.float64) / 0.75))
            x = int(np.searchsorted(c, u[b, d], side="right"))
            assert o["path_nodes"][b, d] == cur and o["out_tokens"][b, d] == x
            nxt = [v for v in range(1, N) if par[b, v] == cur and tok[b, v] == x]
            if not nxt or d == depth:
                break
            cur, d = nxt[0], d + 1
        assert o["accepted_len"][b] == d
        assert (o["path_nodes"][b, d + 1:] == -1).all() and (o["out_tokens"][b, d + 1:] == -1).all()
        lengths.add(d)
    assert len(lengths) >= 3


def pin_sample_edges(lib):
    z = np.full((1, 3, 5), -np.inf, np.float32)
    z[0, 1, 3] = 0.5
    par, tok = np.array([[-1, 0, 1]], np.int32), np.array([[0, 3, 3]], np.int32)
    o = oracle.verify_tree_sample(z, tok, par, [[0.5, 0.5, 0.5]], 1.0, 2, dtype="f32", lib=lib)
    assert o["out_tokens"].tolist() == [[-1, -1, -1]] and o["out_probs"].sum() == 0
    z[0, 0, 3] = -2.0
    o = oracle.verify_tree_sample(z, tok, par, [[0.999, 0.0, 0.5]], 1.0, 2, dtype="f32", lib=lib)
    assert o["path_nodes"].tolist() == [[0, 1, 2]] and o["out_tokens"].tolist() == [[3, 3, -1]]
    # cut at the depth that the call allows; the first of twin children
    z[:] = 0.0
    z[0, 0, 3] = 50.0
    o = oracle.verify_tree_sample(z, [[0, 3, 3]], [[-1, 0, 0]], [[0.5]], 1.0, 0, dtype="f32", lib=lib)
    assert o["accepted_len"].tolist() == [0] and o["out_tokens"].tolist() == [[3]]
    o = oracle.verify_tree_sample(z, [[0, 3, 3]], [[-1, 0, 0]], [[0.5, 0.5]], 1.0, 1, dtype="f32", lib=lib)
    assert o["path_nodes"].tolist() == [[0, 1]]


# ---------------------------------------------------------------------------
# head norms, rotation, cache positions
# ---------------------------------------------------------------------------

def pin_qkv_equals_complex_rotation(lib):
    rng = np.random.default_rng(1)
    B, N, Hq, Hkv, D, L = 2, 5, 3, 2, 8, 20
    qkv = bf16(rng.standard_normal((B, N, Hq + 2 * Hkv, D)))
    qw, kw = bf16(1 + rng.random(D)), bf16(1 + rng.random(D))
    base, depth = np.array([3, 16], np.int32), rng.integers(0, 4, (B, N)).astype(np.int32)
    for inter in (False, True):
        for rot in (8, 4, 0):
            freq = (100.0 ** (-np.arange(rot // 2) / 4)).astype(np.float32)
            q, k, v = oracle.tree_qkv(qkv, qw, kw, 1e-3, freq, base, depth, Hkv, L, 7, inter, lib=lib)
            x = wide(qkv)
            y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-3)
            y[:, :, :Hq] *= wide(qw)
            y[:, :, Hq:] *= wide(kw)
            ang = (7 + base[:, None] - 1 + depth)[:, :, None, None] * freq.astype(np.float64)
            a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
            c = (a + 1j * b) * np.exp(1j * ang)
            want = y.copy()
            if inter:
                want[..., 0:rot:2], want[..., 1:rot:2] = c.real, c.imag
            else:
                want[..., :rot // 2], want[..., rot // 2:rot] = c.real, c.imag
            assert np.allclose(q, want[:, :, :Hq], atol=1e-12)
            for s in range(B):
                at = slice(base[s] - 1, base[s] - 1 + N)
                assert np.allclose(k[s, at], want[s, :, Hq:Hq + Hkv], atol=1e-12)
                assert (v[s, at] == x[s, :, Hq + Hkv:]).all()
                assert np.isnan(k[s, :at.start]).all() and np.isnan(v[s, at.stop:]).all()


def pin_qkv_no_norm_chain(lib):
    qkv = bf16(np.arange(1 * 3 * 3 * 4).reshape(1, 3, 3, 4))
    q, k, v = oracle.tree_qkv(qkv, None, None, 1.0, [np.pi / 2, 0.0], [1], None, 1, 3, lib=lib)
    x = wide(qkv)
    # node 1 of a chain from position 0 turns its first pair by a quarter
    assert np.allclose(q[0, 1, 0], [-x[0, 1, 0, 2], x[0, 1, 0, 1], x[0, 1, 0, 0], x[0, 1, 0, 3]], atol=1e-5)
    assert np.allclose(q[0, 0], x[0, 0, :1]) and (v[0] == x[0, :, 2:]).all()


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------

def pin_attention_equals_dense_softmax(lib):
    rng = np.random.default_rng(2)
    B, N, Hq, Hkv, D, L, P = 2, 6, 4, 2, 8, 25, 5
    q, k, v = (bf16(rng.standard_normal(s)) for s in ((B, N, Hq, D), (B, L, Hkv, D), (B, L, Hkv, D)))
    pk, pv = bf16(rng.standard_normal((P, Hkv, D))), bf16(rng.standard_normal((P, Hkv, D)))
    par = np.stack([synth.make_tree_parents(rng, N) for _ in range(B)]).astype(np.int32)
    base = np.array([1, 14], np.int32)
    mask, _, _ = oracle.tree_mask(par)
    for m in (mask, None):
        for pre in ((None, None), (pk, pv)):
            out, lse = oracle.tree_attention(q, k, v, m, base, 0.3, *pre, lib=lib)
            for b in range(B):
                see = np.zeros((N, L), bool)
                see[:, :base[b] - 1] = True
                for n in range(N):
                    for u in range(N):
                        see[n, base[b] - 1 + u] = u <= n if m is None else (m[b, n, 0] >> u) & 1
                for h in range(Hq):
                    kk, vv, ss = wide(k[b, :, h // 2]), wide(v[b, :, h // 2]), see
                    if pre[0] is not None:
                        kk, vv = np.concatenate([wide(pk[:, h // 2]), kk]), np.concatenate([wide(pv[:, h // 2]), vv])
                        ss = np.concatenate([np.ones((N, P), bool), see], 1)
                    z = np.where(ss, wide(q[b, :, h]) @ kk.T * 0.3, -np.inf)
                    assert np.allclose(out[b, :, h], softmax(z) @ vv, atol=1e-12)
                    assert np.allclose(lse[b, :, h], np.log(np.exp(z).sum(1)), atol=1e-12)


def pin_attention_of_nothing(lib):
    q = bf16(np.ones((1, 2, 1, 4)))
    k = bf16(np.full((1, 3, 1, 4), np.nan))
    k[0, 1] = bf16(np.ones((1, 4)))
    mask = np.array([[[0], [2]]], np.uint32)
    out, lse = oracle.tree_attention(q, k, k, mask, [1], 1.0, lib=lib)
    assert (out[0, 0] == 0).all() and lse[0, 0, 0] == -np.inf
    assert (out[0, 1] == 1).all() and lse[0, 1, 0] == 4.0


PINS = [pin_sample_worked_example, pin_sample_equals_one_by_one_drawing, pin_sample_edges,
        pin_qkv_equals_complex_rotation, pin_qkv_no_norm_chain, pin_attention_equals_dense_softmax,
        pin_attention_of_nothing]

MUTANTS = {
    "sample_last_child": ("for (int v = cur + 1; v < N && child < 0; ++v)", "for (int v = cur + 1; v < N; ++v)"),
    "sample_ignores_parent": ("if (par[v] == cur && tok[v] == x && x >= 0) child = v;", "if (tok[v] == x && x >= 0) child = v;"),
    "sample_root_uniform": ("inverse_cdf(w, V, (double)u[(size_t)b * W + d], &R, &edge)", "inverse_cdf(w, V, (double)u[(size_t)b * W], &R, &edge)"),
    "sample_temperature_dropped": ("exp((logit_at(target, dtype, off + (size_t)j) - m) / T);", "exp(logit_at(target, dtype, off + (size_t)j) - m);"),
    "sample_cut_early": ("if (child < 0 || d == max_depth) break;", "if (child < 0 || d + 1 >= max_depth) break;"),
    "sample_root_row": ("const size_t off = ((size_t)b * N + cur) * (size_t)V;", "const size_t off = ((size_t)b * N) * (size_t)V;"),
    "qkv_no_eps": ("s = 1.0 / sqrt(s / D + eps);", "s = 1.0 / sqrt(s / D);"),
    "qkv_query_weight_for_keys": ("const uint16_t* w = h < Hq ? qn : kn;", "const uint16_t* w = qn;"),
    "qkv_node_number_as_depth": ("(depth ? depth[(size_t)b * N + v] : v)", "v"),
    "qkv_turned_backwards": ("x[a] = xa * cos(t) - xc * sin(t);", "x[a] = xa * cos(t) + xc * sin(t);"),
    "qkv_behind_the_root": ("((size_t)b * L + (size_t)(base[b] - 1 + v)) * Hkv", "((size_t)b * L + (size_t)(base[b] + v - (v > 0))) * Hkv"),
    "qkv_pairs_swapped": ("const int a = interleaved ? 2 * i : i, c = interleaved ? 2 * i + 1 : i + rot / 2;", "const int a = interleaved ? i : 2 * i, c = interleaved ? i + rot / 2 : 2 * i + 1;"),
    "attention_sees_all_nodes": ("            if (!sees) continue;\n", ""),
    "attention_head_by_turns": ("const int hk = h / G;", "const int hk = h % Hkv;"),
    "attention_unscaled": ("s[j] = scale * dot;", "s[j] = dot;"),
    "attention_prefix_short": ("const int u = t - (base[b] - 1);", "const int u = t - base[b];"),
    "attention_lse_without_max": ("cnt ? m + log(total) : -INFINITY;", "cnt ? log(total) : -INFINITY;"),
    "attention_prefix_values_from_cache": ("s[j] * logit_at(j < P ? pv : v, OR_BF16, at[j] + i)", "s[j] * logit_at(v, OR_BF16, at[j] + i)"),
}


@pytest.mark.parametrize("pin", PINS, ids=lambda f: f.__name__[4:])
def test_pin(lib, pin):
    pin(lib)


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_planted_mistake_is_caught(tmp_path, name):
    old, new = MUTANTS[name]
    src = open(SRC).read()
    assert src.count(old) == 1, f"mutation site for {name} not unique/found"
    mutated, lib_path = tmp_path / f"mut_{name}.c", tmp_path / f"libmut_{name}.so"
    mutated.write_text(src.replace(old, new))
    subprocess.run(["gcc", "-O2", "-std=c11", "-fPIC", "-shared", "-o", str(lib_path), str(mutated), "-lm"],
                   check=True)
    variant = oracle.load_variant(str(lib_path))
    for pin in PINS:
        try:
            pin(variant)
        except AssertionError:
            return
    pytest.fail(f"mutant {name} survived every pin")
