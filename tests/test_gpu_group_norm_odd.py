"""Group norm over tokens whose groups are no whole pieces: widths on both sides of every division of a group among lanes."""
import pytest

from tests.test_gpu_group_norm import BF16, F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,C,G", [(700, 63, 1), (700, 65, 1), (700, 1535, 1), (700, 1537, 1), (1200, 1791, 1), (3, 2047, 1), (900, 2047, 1), (900, 2049, 1), (400, 4094, 2),
                                   (400, 4095, 1), (400, 4097, 1), (650, 8955, 5)])
def test_odd_groups(T, C, G, dtype):
    x, w, b, dy = make((1, T), C, dtype, T + C, True, 1 + T % 3)
    check(x, G, w, b, dy, 1, [(0, T)], "token", 32, dtype)


@pytest.mark.parametrize("C,G", [(2048, 1), (4096, 2), (1600, 1)])
def test_rows_an_odd_number_of_elements_apart(C, G):
    """Even groups in rows that begin at odd elements go element by element too."""
    x, w, b, dy = make((1, 700), C + 1, BF16, C, False)
    check(x[..., 1:], G, w, b, dy[..., 1:], 1, [(0, 700)], "token", 32, BF16)
