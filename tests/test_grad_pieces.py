"""How the gradient table cuts its tensors: pieces of at most 32 KB, all of that
but at a tensor's ends."""
import pytest

from padded_permute_combine_gb300 import _lib
from padded_permute_combine_gb300 import build as libbuild

PIECE = 32768


@pytest.mark.parametrize("dtype,size", [(_lib.MOE_F32, 4), (_lib.MOE_BF16, 2)])
@pytest.mark.parametrize("off", [0, 1, 5])
@pytest.mark.parametrize("numel", [1, 8191, 8192, 8193, 16384, 16385, 100003])
def test_pieces_are_whole(numel, off, dtype, size):
    libbuild.build()
    lib = _lib.load()
    entry = (_lib.GradTensor * 1)(_lib.GradTensor((1 << 20) + off * size, None, numel, dtype, 0))
    n = lib.moe_grad_table_pieces(entry, 1)
    pieces = (_lib.GradTensor * n)()
    assert lib.moe_grad_table_fill(entry, 1, pieces, n) == _lib.MOE_OK
    bytes_of = [q.numel * size for q in pieces]
    assert sum(bytes_of) == numel * size and max(bytes_of) <= PIECE
    assert all(b == PIECE for b in bytes_of[1:-1])
    assert n == 1 or bytes_of[0] == PIECE - off * size % 32
