"""s12_gemm_i8 with a few tokens on either side of the sizes at which more warps share a row, against exact integers."""
import pytest

from test_gpu_gemm_i8_few import check, make, s12  # noqa: F401  (s12 is a fixture)
from gpu_util import new_flag

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 2, 5])
@pytest.mark.parametrize("N,K", [(1184, 4112), (1185, 4112), (2368, 4112), (2369, 4112), (4736, 4112), (4737, 1040),
                                 (4737, 12304), (7000, 10384), (7000, 10416), (9475, 2576), (14000, 2624), (3500, 20000)])
def test_rows_shared_by_one_to_eight_warps(s12, M, N, K):  # noqa: F811
    c = make(M, N, K, M + N + K)
    flag = new_flag()
    check(s12.s12_gemm_i8(*c, err_flag=flag, f32=True), *c, True)
    check(s12.s12_gemm_i8(*c, err_flag=flag), *c, False)
    assert int(flag.item()) == 0
