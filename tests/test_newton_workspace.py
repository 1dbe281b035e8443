"""The workspace of the orthogonalised update is what ``zsmr_ops.h`` says: for the
matrices that are worked on at a time 8 bytes an element, and an element of the inner
m x m matrix (m the shorter side) 8, or 20 from a longer side of 1.2 m on; rows are padded to
32 columns."""
import pytest

import zero_sharded_mixed_reduce_amd as z

UP = lambda n: -(-n // 32) * 32     # noqa: E731


@pytest.mark.parametrize("rows,cols", [(129, 129), (300, 150), (1600, 1600), (1600, 1919), (1600, 1920), (1600, 1921), (1920, 1600), (4096, 4096), (4096, 5000),
                                       (300, 360), (104, 129), (1000, 1200), (65, 257), (3, 1000), (14336, 4096), (1, 300)])
@pytest.mark.parametrize("count", [1, 2, 7, 1000, 1 << 20])
def test_bytes_an_element(rows, cols, count):
    m, n = sorted((rows, cols))
    at_a_time = max(1, min(count, (1 << 25) // (m * n)))
    size, each = z.zsmr_orthogonalize_workspace(rows, cols, count), 8 * m * UP(n) + (20 if 5 * n >= 6 * m else 8) * m * UP(m)
    if m * n < 1 << 11:             # 2^14 matrices of few elements at a time at most
        at_a_time = min(at_a_time, 1 << 14)
    # and some sums
    assert 0 <= size - at_a_time * each <= 1 << 18


def test_any_number_of_matrices():
    worst = 0
    for m in [*range(1, 300, 3), *range(300, 5800, 171)]:
        for n in (m, -(-6 * m // 5), 129, 161, 193, 257, 2 * m):
            if n >= m and m * n <= 1 << 25:
                worst = max(worst, z.zsmr_orthogonalize_workspace(m, n, 1 << 20))
    assert 9e8 < worst < 1e9
