"""Lengths that a user gives for a batch reach the library as one 32-bit number per sequence, whatever holds them."""
import numpy as np
import pytest
import torch


def _cache(B):
    import bit_kv_cache_ott_gb300 as pkg
    c = object.__new__(pkg.ByteCache)
    c.B = B
    return c


@pytest.mark.parametrize("lens", [[3, 0, 7, 1], (3, 0, 7, 1), bytes([3, 0, 7, 1]), bytearray([3, 0, 7, 1]), np.array([3, 0, 7, 1]),
                                  np.array([3, 0, 7, 1], np.uint8), torch.tensor([3, 0, 7, 1]), {3: 1, 0: 1, 7: 1, 1: 1}],
                         ids=lambda x: type(x).__name__)
def test_kinds_of_lengths(lens):
    got = _cache(4)._lens(lens)
    assert got.itemsize == 4 and got.tolist() == [3, 0, 7, 1]


class _Short:
    """Says that it holds four, yields three."""

    def __len__(self):
        return 4

    def __iter__(self):
        return iter((1, 2, 3))


@pytest.mark.parametrize("lens", [b"\1\0\0\0\2\0\0\0", [1], [1, 2, 3, 4, 5], _Short(), [1, 2, 3, 2 ** 31], [1, 2, 3, -2 ** 31 - 1]])
def test_refused(lens):
    with pytest.raises(ValueError):
        _cache(4)._lens(lens)


def test_of_another_type():
    with pytest.raises(TypeError):
        _cache(2)._lens([1, 1.5])
    with pytest.raises(TypeError):
        _cache(2)._lens("12")


@pytest.mark.parametrize("pool", [2 ** 31, 2 ** 32 + 8, 2 ** 64 + 8, -2 ** 64 + 8])
def test_blocks_of_a_pool(monkeypatch, pool):
    """A pool is as large as it was asked to be, or refused."""
    import bit_kv_cache_ott_gb300 as pkg
    asked = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(pkg, "load", lambda: type("L", (), {"ott_byte_create": staticmethod(lambda *a: asked.append(a) or -1)}))
    with pytest.raises(ValueError):
        pkg.ByteCache(1, 1, 1, 64, 32, pool_blocks=pool)
    assert not asked
