"""Pins of oracle/mx4_oracle.py against what does not share its code: closed
forms worked by hand from the E2M1 definition, a brute-force nearest-value
search, scale invariants, and a loop-free formulation of the layer in torch."""
import numpy as np
import pytest
import torch

from oracle import mx4_oracle as P
from oracle import mx_oracle as O


@pytest.mark.parametrize("v,code", [
    (0.0, 0x0), (-0.0, 0x8), (0.5, 0x1), (1.0, 0x2), (1.5, 0x3), (2.0, 0x4), (3.0, 0x5),
    (4.0, 0x6), (6.0, 0x7), (-6.0, 0xF),
    (0.25, 0x0),     # halfway 0 / 0.5 -> even code 0
    (0.75, 0x2),     # halfway 0.5 / 1 -> even code 2
    (1.25, 0x2),     # halfway 1 / 1.5 -> even code 2
    (1.75, 0x4),     # halfway 1.5 / 2 -> even code 4
    (2.5, 0x4),      # halfway 2 / 3 -> even code 4
    (3.5, 0x6),      # halfway 3 / 4 -> even code 6
    (5.0, 0x6),      # halfway 4 / 6 -> even code 6
    (5.0001, 0x7), (7.99, 0x7), (-0.2, 0x8), (0.2501, 0x1),
])
def test_e2m1_closed_forms(v, code):
    assert P.e2m1_encode(np.array([v]))[0] == code


def test_encode_is_nearest_by_brute_force():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-8, 8, 4000), np.arange(-64, 65) / 8.0])
    got = P.e2m1_encode(v)
    for x, c in zip(v, got):
        d = np.abs(P.E2M1 - min(abs(x), 6.0))
        near = np.flatnonzero(d == d.min())
        want = near[0] if len(near) == 1 else [n for n in near if n % 2 == 0][0]
        assert c == (want | (8 if np.signbit(x) else 0)), x


def test_scale_rule_and_nonfinite_blocks():
    v = np.zeros((6, 32))
    v[1, 3] = 1.0            # X = -2: the value becomes 4
    v[2, 0] = -7.9           # X = 0: saturates at 6
    v[3, 5] = 2.0 ** -133    # X clamped to -127
    v[4, 9] = np.inf
    v[5, 1] = np.nan
    codes, scales = P.quantize4_lastdim(v)
    assert scales[:, 0].tolist() == [0, 125, 127, 0, 255, 255]
    c = P.unpack(codes)
    assert c[1, 3] == 6 and c[2, 0] == 0xF and c[3, 5] == 0
    assert not c[4].any() and not c[5].any()
    back = P.dequantize4_lastdim(codes, scales)
    assert back[1, 3] == 1.0 and back[2, 0] == -6.0
    assert np.isnan(back[4]).all() and np.isnan(back[5]).all()


def test_representable_values_survive_and_amax_is_kept_below_eight_scales():
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16, (50, 32))
    c[:, 0] = rng.choice([6, 7, 14, 15], 50)           # amax 4 or 6: X as built
    X = rng.integers(-100, 100, 50)
    v = P.e2m1_decode(c) * np.ldexp(1.0, X)[:, None]
    codes, scales = P.quantize4_lastdim(v)
    assert np.array_equal(P.unpack(codes), c) and np.array_equal(scales[:, 0], X + 127)
    w = rng.standard_normal((200, 64)) * np.exp(rng.uniform(-20, 20, (200, 1)))
    _, s = P.quantize4_lastdim(w)
    amax = np.abs(w.reshape(200, 2, 32)).max(-1)
    two = np.ldexp(1.0, s.astype(int) - 127)
    assert (4 * two <= amax).all() and (amax < 8 * two).all()


def test_route_masks_and_ties():
    inf = np.inf
    lg = np.array([[1.0, 1.0, 1.0, 0.0], [-inf, 2.0, -inf, -inf], [-inf] * 4,
                   [np.nan, 0.0, 3.0, -inf]])
    ids, r = P.route(lg, 2)
    assert ids[0].tolist() == [0, 1] and np.allclose(r[0], 0.5)
    assert ids[1, 0] == 1 and r[1].tolist() == [1.0, 0.0]
    assert r[2].tolist() == [0.0, 0.0]
    assert ids[3].tolist() == [2, 1] and np.allclose(r[3], [1 / (1 + np.exp(-3)), 1 / (1 + np.exp(3))])


@pytest.mark.parametrize("mx", [False, True])
def test_layer_against_a_dense_torch_formulation(mx):
    rng = np.random.default_rng(3)
    T, E, k, H, F = 5, 6, 3, 64, 32
    x = O.round_bf16(rng.standard_normal((T, H)))
    w1, w2 = rng.standard_normal((E, 2 * F, H)) * 0.2, rng.standard_normal((E, H, F)) * 0.2
    lg = rng.standard_normal((T, E))
    lg[3] = -np.inf
    got = P.moe_layer(x, lg, w1, w2, k, mx)
    xt = torch.from_numpy(O.qdq_lastdim(x) if mx else x)
    top = torch.topk(torch.from_numpy(lg), k, dim=1)
    r = torch.zeros(T, E, dtype=torch.float64)
    r[:3] = r[:3].scatter(1, top.indices[:3], torch.softmax(top.values[:3], 1))
    r[4:] = r[4:].scatter(1, top.indices[4:], torch.softmax(top.values[4:], 1))
    h = torch.einsum("th,efh->tef", xt, torch.from_numpy(w1))
    z = r[..., None] * torch.nn.functional.silu(h[..., :F]) * h[..., F:]
    z = torch.from_numpy(O.qdq_lastdim(z.numpy()) if mx else O.round_bf16(z.numpy()))
    want = torch.einsum("tef,ehf->th", z, torch.from_numpy(w2)).numpy()
    assert not got[3].any()
    # equal up to the rare code that the two summation orders round apart
    assert np.linalg.norm(got - want) <= 1e-6 * np.linalg.norm(want)
