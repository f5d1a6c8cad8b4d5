"""Host-side tests (no GPU needed) of the bytes that kda_logits_process's buffers span:
what its overlap checks compare. Addresses are compared only."""
import pytest

from test_host_linear_logits import ALIAS, INVALID, LISTS, OK, err, logits

FP32, FAR = 0, 1 << 63


def call(lib, rows, stride, at, **kw):
    """out at 4096, rows of 64 logits `stride` apart; everything else above 2^63 but `at`."""
    far = {n: FAR + (i + 1 << 56) for i, n in enumerate(LISTS)}
    args = dict(rows=rows, vocab=64, dtype=FP32, logits=FAR, row_stride=64, out=4096, out_stride=stride, token_stride=0,
                bias_stride=0, allowed_stride=0)
    return logits(lib, **{**args, **far, **at, **kw})


@pytest.mark.parametrize("rows,stride", [(3, 1 << 40), ((1 << 20) - 1, 1 << 40), (1 << 22, 1 << 38),
                                         ((1 << 23) - 1, (1 << 37) - 1)])
def test_overlaps_far_behind_the_first_row_are_found(kda_lib, rows, stride):
    last = 4096 + 4 * (rows - 1) * stride
    assert call(kda_lib, rows, stride, {}) == OK, err(kda_lib)
    for at in (4096 + 4 * stride, last, last + 4 * 63):
        assert call(kda_lib, rows, stride, dict(tokens=at)) == ALIAS, at
    assert call(kda_lib, rows, stride, dict(tokens=last + 4 * 64)) == OK, err(kda_lib)


@pytest.mark.parametrize("rows,stride", [((1 << 22) + 1, 1 << 40), ((1 << 23) - 1, 1 << 40), ((1 << 21) + 1, 1 << 40),
                                         ((1 << 23) - 1, 1 << 38), ((1 << 20) + 1, 1 << 40)])
def test_rows_that_pass_64_bits_are_refused(kda_lib, rows, stride):
    """In 64 bits, 2^22 rows of 2^40 fp32 logits span nothing but the last row: row 1 in front of a list was not seen."""
    assert call(kda_lib, rows, stride, dict(tokens=4096 + 4 * stride)) == INVALID
    for name in ("row_stride", "token_stride", "bias_stride", "allowed_stride"):
        assert call(kda_lib, rows, 64, {}, **{name: stride}) == INVALID, name
    assert call(kda_lib, rows, 64, {}) == OK, err(kda_lib)
