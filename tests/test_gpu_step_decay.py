"""A decay's error enters the state once a token, and does not cancel where it is of one sign.  The typical error of the
states (root mean square over all columns, relative to their size) is at most twice that of the recurrence taken in FP32 by
NumPy, which rounds as often: room for sums in another order, none for decays of fewer bits."""
import numpy as np
import pytest
import torch

from tests.step_testutil import f64
from tests.test_gpu_step import make, run
from tests.test_gpu_step_precision import measures, recurrence

pytestmark = pytest.mark.gpu


def check(x, kda, states):
    exact, plain = recurrence(x, kda), recurrence(x, kda, np.float32)
    got, ref = measures(x, kda, exact, f64(states)), measures(x, kda, exact, plain[1])
    assert got[0] <= 1 and got[1] <= 2 * ref[1], (got, ref)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("lens,H,HV", [([20, 17, 22], 1, 3), ([20, 23], 13, 39), ([11] * 20, 4, 16), ([256], 2, 6),
                                       ([150, 90], 13, 52)], ids=str)
def test_one_call(lens, H, HV, kda):
    x = make(lens, H, HV, len(lens), "fp32", kda, seed=sum(lens) + HV + kda)
    _, pool, status = run(x, kda, None, None)
    assert status == 0
    check(x, kda, pool)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("N,H,HV", [(2, 2, 4), (3, 8, 24), (1, 10, 40)])
def test_token_by_token(N, H, HV, kda):
    import linear_attention_gdn_gb300 as gdn
    L = 200
    x = make([L] * N, H, HV, N, "fp32", kda, seed=N + HV + kda)
    pool, err = x["states"].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    d = {n: x[n].unflatten(0, (N, L)).transpose(0, 1).contiguous().cuda() for n in ("q", "k", "v", "g", "beta")}
    o, prob = torch.empty((N, HV, 128), device="cuda"), gdn.step_problem(N, N, H, HV, N, dtype=torch.float32)
    for t in range(L):
        (gdn.gdn_kda_step if kda else gdn.gdn_step)(prob, *(d[n][t] for n in ("q", "k", "v", "g", "beta")), pool, o, err)
    assert gdn.gdn_device_status(err) == 0
    check(x, kda, pool)
