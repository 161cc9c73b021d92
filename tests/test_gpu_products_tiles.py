"""The grouped and fp8 products by tile: every kernel, every split of a contraction and every number of scale blocks
that the choice of tiles reaches, against the formula in 64 bits; and every kernel with its producers' waits made to
run out."""
import pytest
import torch

from grouped_cases import CASES, GROUPED, LONG, Operands, case_id, plan

pytestmark = pytest.mark.gpu

rmm = pytest.importorskip("input_adaptive_reduced_colnorm_b200")


@pytest.fixture(scope="module", autouse=True)
def built():
    from input_adaptive_reduced_colnorm_b200 import build
    build.build()
    yield
    assert rmm.device_error() == 0


@pytest.mark.parametrize("case", CASES, ids=case_id)
def test_tile(case):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    o = Operands(case)
    assert plan(o.dtype, o.n, o.d, o.m, o.groups, sms) == case[4]
    out = o.out()
    o.call(out)
    o.check(out, *o.reference())
    behind = out.as_strided((o.n, out.stride(0)), (out.stride(0), 1))[:, o.m:]
    assert behind.isnan().all()  # the buffer's columns past m are as they were
    again = o.out()
    o.call(again)
    assert torch.equal(again, out)  # the same result every time


TIMEOUT_PRODUCER = 1


@pytest.mark.parametrize("case", LONG, ids=case_id)
def test_expired_wait_returns_and_leaves_the_context_usable(case):
    """Producers that stop after their first stages: the other roles leave their waits, the kernel returns with the
    producer's code, writes nothing outside the groups' rows, and the next call is right."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    o = Operands(case)
    assert plan(o.dtype, o.n, o.d, o.m, o.groups, sms) == case[4]
    assert rmm.device_error() == 0
    out = o.out()
    assert o.expire(out) == 0, rmm.lib().rmm_last_error()
    torch.cuda.synchronize()
    assert rmm.device_error() == TIMEOUT_PRODUCER
    assert rmm.device_error() == 0  # the read cleared it
    assert (out[: o.before] == 3).all() and (out[o.n - o.behind:] == 3).all()
    behind = out.as_strided((o.n, out.stride(0)), (out.stride(0), 1))[:, o.m:]
    assert behind.isnan().all()
    o.call(out)
    o.check(out, *o.reference())
    assert rmm.device_error() == 0


@pytest.mark.parametrize("case", GROUPED, ids=case_id)
def test_nan_stays_in_its_rows_and_its_group(case):
    """NaN and infinity in rows of no group, in the weights (and their scales) of a group without rows, in the first
    row of each second group that has rows, just past the end of another one (in its values, or for e4m3 in the scale
    of its last block), and in the scale of row 0: only the rows that hold them are NaN."""
    o = Operands(case)
    ref, mag = o.reference()
    nan, t = float("nan"), o.X.dtype
    sick = torch.zeros(o.n, dtype=torch.bool, device="cuda")
    with_rows = [e for e in range(o.groups) if o.bounds[e + 1] > o.bounds[e]]
    for k, e in enumerate(with_rows[1::2]):
        row = o.bounds[e]
        sick[row] = True
        if o.dtype and k % 2:
            o.sx[-1, row] = nan
        else:
            o.X[row, o.d - 1] = torch.tensor(nan).to(t)
    for e in range(o.groups):
        if e not in with_rows:
            o.W[e] = torch.tensor(nan).to(t)
            if o.dtype:
                o.sw[e] = nan
    o.X[: o.before] = torch.tensor(nan).to(t)
    o.X[o.n - o.behind:] = torch.tensor(nan).to(t)
    if o.dtype:
        o.sx[:, : o.before] = nan
        o.sx[:, o.n - o.behind:] = float("inf")
    out = o.out()
    o.call(out)
    assert out[sick].isnan().all()
    o.check(out, ref, mag, ~sick)
