"""How much workspace the block-scaled forward asks for, without a GPU.  Every call here is stopped by a later argument
check (x is missing), so none reaches the device."""

import pytest

import fp8_delayed_scaling_amax_b200 as F

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5


def _forward(m, k, n, fp8, w8_out=False, x8c_out=False, work=None, nbytes=0):
    """The call with neither x nor y: what refuses it."""
    rc = F.lib().linear_forward_fp8_block(None, 512, int(fp8), 4096 if fp8 else None, None, m, k, n, 0,
                                          8192 if w8_out else None, 4096 if w8_out else None, 8192 if x8c_out else None,
                                          4096 if x8c_out else None, work, nbytes, None, None)
    return rc, F.last_error()


def _x_part(m, k):
    return F.linear_forward_fp8_block_workspace_size(m, k, 0)


def test_the_size_without_a_weight_is_that_of_x():
    for m, k in ((1, 16), (17, 4096), (300, 1040), (2048, 1024)):
        part = _x_part(m, k)
        assert part % 256 == 0 and m * k + 4 * m * -(-k // 128) <= part <= m * k + 4 * m * -(-k // 128) + 2 * 255
        assert part < F.linear_forward_fp8_block_workspace_size(m, k, 8192) - 8192 * k


@pytest.mark.parametrize("m", [1, 16])
@pytest.mark.parametrize("fp8,w8_out", [(True, False), (False, True)])
def test_a_few_rows_need_no_workspace(m, fp8, w8_out):
    rc, why = _forward(m, 8192, 8192, fp8, w8_out)
    assert rc == INVALID and why.startswith("x, w and y")
    # the column form of x is wanted: x is quantized by a launch of its own
    rc, why = _forward(m, 8192, 8192, fp8, w8_out, x8c_out=True)
    assert rc == INVALID and why.startswith("workspace")


@pytest.mark.parametrize("m", [1, 17, 300])
@pytest.mark.parametrize("fp8,w8_out", [(True, False), (False, True)])
def test_a_weight_kept_elsewhere_takes_no_workspace(m, fp8, w8_out):
    k, n, columns = 1040, 4096, m <= 16
    part = _x_part(m, k)
    rc, why = _forward(m, k, n, fp8, w8_out, columns, 1024, part)
    assert rc == INVALID and why.startswith("x, w and y")
    assert _forward(m, k, n, fp8, w8_out, columns, 1024, part - 1)[0] == WORKSPACE
    assert _forward(m, k, n, fp8, w8_out, columns, 1040, part)[0] == UNSUPPORTED
    rc, why = _forward(m, k, n, fp8, w8_out, columns)
    assert rc == INVALID and why.startswith("workspace")


@pytest.mark.parametrize("m", [1, 17, 300])
@pytest.mark.parametrize("fp8", [False, True])
def test_no_columns_of_the_weight_need_no_workspace(m, fp8):
    """Without outputs there is nothing to do, unless x's column form is wanted."""
    rc, why = _forward(m, 1040, 0, fp8)
    assert rc == INVALID and why.startswith("x, w and y")
    rc, why = _forward(m, 1040, 0, fp8, x8c_out=True)
    assert rc == INVALID and why.startswith("workspace")


@pytest.mark.parametrize("m", [1, 16, 17, 300])
def test_a_weight_quantized_in_the_call_takes_all_of_it(m):
    k, n = 1040, 4096
    need = F.linear_forward_fp8_block_workspace_size(m, k, n)
    rc, why = _forward(m, k, n, False, work=1024, nbytes=need)
    assert rc == INVALID and why.startswith("x, w and y")
    assert _forward(m, k, n, False, work=1024, nbytes=need - 1)[0] == WORKSPACE
    assert _forward(m, k, n, False)[0] == INVALID
