"""Queries, keys and values that are broadcast along a dimension, without a GPU: they
hold fewer rows than their shape says, so no stride between tokens describes them."""
import pytest

from tests.test_cache_checks import APPEND_OK, ATTEND_OK, b16, i64, stub  # noqa: F401


@pytest.mark.parametrize("q", [
    b16(3, 1, 4, 64).expand(3, 5, 4, 64),    # one token of each sequence, repeated
    b16(1, 5, 4, 64).expand(3, 5, 4, 64),    # one sequence, repeated
    b16(1, 1, 4, 64).expand(3, 5, 4, 64),
    b16(3, 1, 8, 64)[:, :, 2:6].expand(3, 5, 4, 64),
    b16(3, 5, 1, 64).expand(3, 5, 4, 64),    # one head, repeated
    b16(3, 5, 4, 1).expand(3, 5, 4, 64)])
def test_queries(stub, q):  # noqa: F811
    with pytest.raises(ValueError):
        ATTEND_OK(q=q)
    assert stub.calls == []


@pytest.mark.parametrize("rows", [
    b16(3, 1, 2, 64).expand(3, 5, 2, 64), b16(1, 5, 2, 64).expand(3, 5, 2, 64), b16(1, 1, 2, 64).expand(3, 5, 2, 64),
    b16(3, 1, 1, 2, 64).expand(3, 1, 5, 2, 64), b16(3, 1, 9, 64)[:, :, 4:6].expand(3, 5, 2, 64)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_keys_and_values(stub, what, rows):  # noqa: F811
    whole = b16(15, 2, 64)
    with pytest.raises(ValueError):
        APPEND_OK(**{"k": whole, "v": whole, "slots": i64(15), what: rows})
    assert stub.calls == []


def test_dimensions_of_one_may_have_any_stride(stub):  # noqa: F811
    ATTEND_OK(q=b16(3, 1, 4, 64).expand(3, 1, 4, 64))
    ATTEND_OK(q=b16(3, 9, 64)[:, None, 2:6])
    ATTEND_OK(q=b16(3, 5, 9, 64)[:, :1, 2:6])
    APPEND_OK(k=b16(7, 1, 9, 64)[:, :, 2:4], v=b16(1, 7, 9, 64)[:, :, 2:4])
    assert [args[1]._obj.q_stride for _, args in stub.calls[:3]] == [256, 9 * 64, 45 * 64]
    assert len(stub.calls) == 4 and stub.calls[3][1][2] == stub.calls[3][1][4] == 9 * 64
