"""Which rows with a pitch overlap (CPU only: the check is ahead of any CUDA call), against a search element by element."""
import pytest

torch = pytest.importorskip("torch")

from megatron_tensor_mlp_gb300 import build as B  # noqa: E402

B.build()
from megatron_tensor_mlp_gb300 import tpmlp as T  # noqa: E402

BASE, ES = 0x7F0000000000, 2
REACHED = (T.OK, T.ERR_CUDA, T.ERR_ARCH)


def norm(x, y, rows, h, ldx, ldy):
    return T.tpmlp_layernorm_fwd(BASE + x * ES, None, None, BASE + y * ES, None, None, rows, h, ldx, ldy, stream=0, check=False)


def norm_bwd(x, dy, dx, rows, h, ld):
    far = BASE + (1 << 30)
    return T.tpmlp_layernorm_bwd(BASE + x * ES, None, far, far + 4096, BASE + dy * ES, BASE + dx * ES, None, None, None, rows, h, ld, ld, ld,
                                 stream=0, check=False)


def test_columns_of_one_tensor_are_not_an_overlap():
    """x, and what is made of it, as neighbouring columns of one tensor of a pitch."""
    assert norm(0, 64, 16, 64, 128, 128) in REACHED
    assert norm(64, 0, 16, 64, 128, 128) in REACHED
    assert norm_bwd(0, 64, 128, 16, 64, 192) in REACHED
    assert norm_bwd(128, 64, 0, 16, 64, 256) in REACHED


def test_rows_of_equal_pitch_against_their_elements():
    for rows in (1, 2, 5):
        for h, ld in ((1, 1), (3, 3), (3, 4), (3, 6), (4, 9), (5, 8)):
            own = {r * ld + i for r in range(rows) for i in range(h)}
            for y in range(3 * ld * rows):
                meet = any(y - rows * ld + e in own for e in own)
                st = norm(rows * ld, y, rows, h, ld, ld)
                assert (st == T.ERR_ALIAS) == meet, (rows, h, ld, y, st)


def test_rows_of_other_pitches_are_refused_where_their_ranges_meet():
    assert norm(0, 64, 16, 64, 128, 192) == T.ERR_ALIAS
    assert norm(0, 16 * 128, 16, 64, 128, 192) in REACHED
