"""Which outputs of the calls between a block's linears the binding takes for
overlapping (no GPU: only addresses and strides count)."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S


def _bytes(t):
    n = t.element_size()
    out = set()
    for at in itertools.product(*(range(s) for s in t.shape)):
        first = t.data_ptr() + n * sum(i * s for i, s in zip(at, t.stride()))
        out.update(range(first, first + n))
    return out


def _refused(a, b) -> bool:
    try:
        S._refuse_overlaps((("a", a),), (("b", b),))
    except ValueError as e:
        assert str(e) == "a: overlaps b"
        return True
    return False


def test_against_every_byte():
    base = torch.zeros(4000, dtype=torch.int16)
    gen = torch.Generator().manual_seed(1)
    pick = lambda n: int(torch.randint(0, n, (1,), generator=gen))   # noqa: E731
    met = 0
    for _ in range(600):
        pair = []
        for _ in range(2):
            shape = [1 + pick(3), 1 + pick(4), pick(4) if pick(20) == 0 else 1 + pick(3), 4]
            strides = [1 + pick(500), 1 + pick(100), 1 + pick(40), 1]
            pair.append(base.as_strided(shape, strides, pick(1500)))
        want = bool(_bytes(pair[0]) & _bytes(pair[1]))
        assert _refused(*pair) == want and _refused(*pair[::-1]) == want
        met += want
    assert 50 < met < 550   # both kinds


def test_slices_of_one_buffer():
    qkv = torch.zeros(2, 7, 5, 8, dtype=torch.bfloat16)
    q, k, v = qkv.split([3, 1, 1], 2)
    assert not _refused(q, k) and not _refused(k, v) and _refused(q, qkv) and _refused(q, q[:, 3:4])
    assert not _refused(q[:, :3], q[:, 3:]) and _refused(q[:, :4], q[:, 3:]) and not _refused(q[:, :0], q)
    S._refuse_overlaps((("dq", q), ("dk", k), ("dv", v)), (("q", torch.zeros_like(q)), ("mask", None)))
    with pytest.raises(ValueError, match="dq: overlaps k"):
        S._refuse_overlaps((("dq", q),), (("k", qkv[:, :, 2:4]),))
    with pytest.raises(ValueError, match="dk: overlaps dv"):
        S._refuse_overlaps((("dq", q), ("dk", v), ("dv", v)), ())
    # an input itself, not a part of it or its memory in another order
    x = torch.zeros(6, 6)
    S._refuse_overlaps((("s", x),), (), (("x", x), ("h", x.view(6, 6))))
    for other in (x.t(), x[:5], x.view(4, 9)):
        with pytest.raises(ValueError, match="is not x itself"):
            S._refuse_overlaps((("s", other),), (), (("x", x),))
    one = torch.zeros(1, 9)   # (a dimension of one may have any stride)
    S._refuse_overlaps((("s", one.as_strided((1, 9), (50, 1))),), (), (("x", one),))
