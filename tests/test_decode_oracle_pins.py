"""Pins of the decoding operators' oracle: hand-worked values and independent routes, so
that the GPU tests compare against something that was itself checked."""
import numpy as np
import pytest

from oracle import decode_oracle as do


def _cache(rng, lens, Hkv=2, page=16, C=64, spare=2):
    need = [-(-n // page) for n in lens]
    P = sum(need) + spare
    order = rng.permutation(P - spare) if P > spare else np.array([], int)
    table = np.full((len(lens), max(1, max(need))), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return dict(k=rng.standard_normal((P, Hkv, page, C)), v=rng.standard_normal((P, Hkv, page, C)),
                acc=rng.gamma(0.5, size=(P, Hkv, page)), ordinal=np.zeros((P, Hkv, page), np.int64),
                table=table, lens=np.array(lens), k_scale=None, v_scale=None)


def test_rope_quarter_turns():
    # one pair per axis, a quarter turn per position: (x1, x2) -> (-x2, x1) -> (-x1, -x2)
    x = np.zeros((1, 1, 3, 64))
    x[..., :4] = [3.0, 7.0, 5.0, 11.0]
    pos = np.array([[[0, 2], [1, 0], [2, 1]]])
    y = do.rope(x, pos, [np.pi / 2, np.pi / 2], (1, 1))
    # halves: pair 0 = elements (0, 2) on axis 0, pair 1 = elements (1, 3) on axis 1
    np.testing.assert_allclose(y[0, 0, 0, :4], [3, -7, 5, -11], atol=1e-12)
    np.testing.assert_allclose(y[0, 0, 1, :4], [-5, 7, 3, 11], atol=1e-12)
    np.testing.assert_allclose(y[0, 0, 2, :4], [-3, -11, -5, 7], atol=1e-12)
    # interleaved: pair 0 = elements (0, 1), pair 1 = (2, 3)
    y = do.rope(x, pos, [np.pi / 2, np.pi / 2], (1, 1), interleaved=True)
    np.testing.assert_allclose(y[0, 0, 1, :4], [-7, 3, 5, 11], atol=1e-12)
    np.testing.assert_allclose(y[0, 0, 2, :4], [-3, -7, -11, 5], atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_and_its_inverse_is_its_gradient(interleaved):
    rng = np.random.default_rng(0)
    x, g = rng.standard_normal((2, 1, 2, 5, 64))
    pos = rng.integers(0, 1000, (1, 5, 2))
    f = rng.uniform(0, 1, 24)
    y = do.rope(x, pos, f, (8, 16), interleaved)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
    np.testing.assert_allclose(do.rope(y, pos, f, (8, 16), interleaved, inverse=True), x, atol=1e-12)
    grad = do.rope(g, pos, f, (8, 16), interleaved, inverse=True)
    eps = 1e-6
    for i in range(0, 64, 7):     # differences of <g, rope(x)>
        d = np.zeros_like(x)
        d[0, 1, 3, i] = eps
        num = ((do.rope(x + d, pos, f, (8, 16), interleaved) -
                do.rope(x - d, pos, f, (8, 16), interleaved)) * g).sum() / (2 * eps)
        assert abs(num - grad[0, 1, 3, i]) < 1e-7


def test_append_then_rows_gives_the_tokens_back():
    rng = np.random.default_rng(1)
    c = _cache(rng, [20, 3, 0])
    k, v = rng.standard_normal((2, 3, 2, 5, 64))
    out = do.cache_append(c, k, v, [5, 2, 0], [120, 3, 0])
    np.testing.assert_array_equal(do.cache_rows(out, "k", 0, 1)[15:], k[0, 1])
    np.testing.assert_array_equal(do.cache_rows(out, "v", 1, 0)[1:], v[1, 0, :2])
    np.testing.assert_array_equal(do.cache_rows(out, "k", 1, 0)[:1], do.cache_rows(c, "k", 1, 0)[:1])
    assert [int(x) for x in do.cache_rows(out, "ordinal", 0, 0)[15:]] == [115, 116, 117, 118, 119]
    assert (do.cache_rows(out, "acc", 0, 0)[15:] == 0).all()


def test_decode_against_torch_attention_and_closed_forms():
    import torch
    rng = np.random.default_rng(2)
    c = _cache(rng, [37, 0, 1], C=64)
    q = rng.standard_normal((3, 4, 64))
    o, lse, w = do.decode_attention(q, c, 0.125)
    k = np.stack([do.cache_rows(c, "k", 0, h) for h in range(2)])
    v = np.stack([do.cache_rows(c, "v", 0, h) for h in range(2)])
    t = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[0])[:, None], torch.from_numpy(np.repeat(k, 2, 0)),
        torch.from_numpy(np.repeat(v, 2, 0)), scale=0.125)
    np.testing.assert_allclose(o[0], t[:, 0].numpy(), atol=1e-12)
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()
    np.testing.assert_allclose(o[2, 3], do.cache_rows(c, "v", 2, 1)[0], atol=1e-12)  # one key
    assert abs(w[0][0].sum() - 2) < 1e-12                     # two query heads per kv head
    o0, lse0, w0 = do.decode_attention(0 * q, c, 0.125)       # equal weights
    np.testing.assert_allclose(o0[0, 0], v[0].mean(0), atol=1e-12)
    assert abs(lse0[0, 0] - np.log(37)) < 1e-12


def test_evict_by_hand():
    # slots:     0    1    2    3    4    5
    acc = [0.1, 0.9, 0.5, 0.5, 0.0, 0.7]
    age = [0, 1, 2, 3, 4, 5]
    assert do.evict_kept(acc, age, 3, 6, 0, 0) == {1, 5, 2}          # tie 2 / 3: the lower slot
    assert do.evict_kept(acc, age, 3, 6, 2, 0) == {4, 5, 1}          # the two last are safe
    assert do.evict_kept(acc, age, 3, 6, 1, 1) == {0, 5, 1}          # the first and the last
    assert do.evict_kept(acc, [5, 4, 3, 2, 1, 0], 2, 6, 1, 0) == {0, 1}   # by ordinal, not by slot
    assert do.evict_kept([0.1, np.nan, np.inf, 2], [0, 1, 2, 3], 2, 4, 0, 0) == {1, 2}
    rng = np.random.default_rng(3)
    c = _cache(rng, [6], Hkv=1, C=64)
    pg = c["table"][0, 0]
    c["acc"][pg, 0, :6], c["ordinal"][pg, 0, :6] = acc, age
    out = do.cache_evict(c, 3, 0, 0, [6])
    # kept {1, 2, 5}: hole 0 takes slot 5
    np.testing.assert_array_equal(do.cache_rows(out, "k", 0, 0), c["k"][pg, 0, [5, 1, 2]])
    np.testing.assert_array_equal(do.cache_rows(out, "ordinal", 0, 0), [5, 1, 2])
    # two holes: the first takes the LAST kept slot
    c["acc"][pg, 0, :6] = [0, 9, 0, 1, 8, 7]
    out = do.cache_evict(c, 3, 0, 0, [6])
    np.testing.assert_array_equal(do.cache_rows(out, "ordinal", 0, 0), [5, 1, 4])
    np.testing.assert_array_equal(out["k"][pg, 0, 3:], c["k"][pg, 0, 3:])      # slots from n on


def test_attention_after_evicting_nothing_heavy():
    """Dropping slots of zero weight changes no output: eviction and attention agree on
    which rows are which."""
    rng = np.random.default_rng(4)
    c = _cache(rng, [40], Hkv=1, C=64)
    far = rng.choice(40, 15, replace=False)
    for s in far:
        pg, r = do.cache_slot(c, 0, int(s))
        c["k"][pg, 0, r] = -50.0 * np.ones(64)
    q = np.abs(rng.standard_normal((1, 2, 64))) + 0.5
    o, lse, w = do.decode_attention(q, c, 0.125)
    for s in range(40):
        pg, r = do.cache_slot(c, 0, s)
        c["acc"][pg, 0, r] = w[0][0][s]
    out = do.cache_evict(c, 25, 0, 0, [40])
    o2, lse2, _ = do.decode_attention(q, out, 0.125)
    np.testing.assert_allclose(o2, o, atol=1e-12)
    np.testing.assert_allclose(lse2, lse, atol=1e-12)
