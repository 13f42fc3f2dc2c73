"""Pins of the attention-layer oracle."""
import numpy as np
import pytest

from oracle import attn as oa


def test_e4m3_table_and_rounding_against_torch():
    import torch
    t = oa.e4m3_table()
    ref = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t, ref.astype(np.float64), equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-4, 3, 4000), t[:127], [0.0, -0.0, 448, 449, 1e9],
                        (t[:126] + t[1:127]) / 2])          # ties among them
    x = x.astype(np.float32)
    got = oa.quantize_e4m3(x[None], None)[0]
    want = torch.tensor(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 32)).astype(np.float32)
    freq = 10.0 ** -rng.uniform(0, 3, 8)
    y = oa.norm_rope(x, None, freq, 100000, [0, 1, 1], 1e-6, interleaved=interleaved)
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * np.array([100000, 100001, 100001])[:, None, None] * freq)
    assert np.allclose(y[..., a], z.real, atol=1e-9) and np.allclose(y[..., b], z.imag, atol=1e-9)
    assert np.array_equal(y[..., 16:], x[..., 16:].astype(np.float64))


def test_norm_of_a_constant_head():
    x = np.full((1, 1, 16), 3.0, dtype=np.float32)
    y = oa.norm_rope(x, np.full(16, 0.5, dtype=np.float32), [], 0, [0], 0.0, offset=1.0)
    assert np.allclose(y, 1.5)


def _small(rng, T, Hq, Hkv, d, n, S):
    P = max(1, -(-n // S))
    pages = rng.permutation(P + 2)[:P].astype(np.int32)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    return f(T, Hq, d), f(T, Hkv, d), f(T, Hkv, d), f(P + 2, Hkv, S, d), f(P + 2, Hkv, S, d), pages


def test_one_slot_is_its_value_and_no_slot_is_zero():
    rng = np.random.default_rng(2)
    q, k, v, kc, vc, pages = _small(rng, 1, 2, 1, 16, 0, 16)
    assert np.allclose(oa.attn_span(q, k, v, kc, vc, pages, 0), v[:, [0, 0]])


def test_uniform_scores_give_the_mean():
    rng = np.random.default_rng(3)
    q, k, v, kc, vc, pages = _small(rng, 1, 1, 1, 16, 20, 16)
    out = oa.attn_span(q * 0, k, v, kc, vc, pages, 20)
    rows = np.concatenate([vc[pages[0], 0], vc[pages[1], 0, :4], v[:, 0]])
    assert np.allclose(out[0, 0], rows.mean(0))
    pages[0] = -1
    rows = rows[16:]
    assert np.allclose(oa.attn_span(q * 0, k, v, kc, vc, pages, 20)[0, 0], rows.mean(0))
    out = oa.attn_span(q * 0, k, v, kc, vc, pages, 20, window=3)
    assert np.allclose(out[0, 0], rows[-3:].mean(0))


def test_tree_node_equals_chain_over_its_root_path():
    rng = np.random.default_rng(4)
    q, k, v, kc, vc, pages = _small(rng, 6, 4, 2, 16, 37, 16)
    parent = [-1, 0, 0, 1, 2, 3]
    for window in (0, 2, 9):
        tree = oa.attn_span(q, k, v, kc, vc, pages, 37, parent=parent, window=window)
        for path in ([0, 1, 3, 5], [0, 2, 4]):
            ch = oa.attn_span(q[path], k[path], v[path], kc, vc, pages, 37, window=window)
            assert np.allclose(tree[path], ch)


def test_append_places_rows():
    rows = np.arange(5 * 2 * 16, dtype=np.uint16).reshape(5, 2, 16)
    cache = np.zeros((3, 2, 16, 16), dtype=np.uint16)
    oa.append(rows, cache, [2, 7, 0], 14, [0, 3, 4, -1], 3)
    assert np.array_equal(cache[2, :, 14], rows[0]) and np.array_equal(cache[2, :, 15], rows[3])
    assert not cache[0].any() and not cache[1].any()      # page 7 is not there: row 4 is not written
