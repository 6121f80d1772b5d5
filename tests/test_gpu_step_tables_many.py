"""The tables of a generation step for the most requests: at, and past, what a CTA keeps of them in shared memory (8,192)."""
import numpy as np
import pytest

from tests.test_gpu_step_tables import books, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N", [8191, 8192, 8193, 16384])
@pytest.mark.parametrize("hi", [1, 9])
def test_many_requests(N, hi, in_place):
    """All fit, some have ended; tokens by the second kernel."""
    b = books(N, 4, 8, 20, spare=3 * N, seed=N + hi, done=N // 7, hi=hi)
    T = int(np.maximum(b[0], 0).sum())
    assert T > 2048
    run(*b, T=T + 3, block=4, in_place=in_place, offset=int(in_place))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N", [8192, 8193, 16384])
def test_few_tokens_of_many_requests(N, in_place):
    """Up to 2,048 tokens the first kernel writes theirs itself: it reads the contexts again while others' are written."""
    lengths, *rest = books(N, 4, 8, 20, spare=N, seed=N, done=0, hi=5)
    takes = np.random.default_rng(N).permutation(N)
    lengths[takes[300:]] = 0
    lengths[takes[300:700]] = -1
    T = int(np.maximum(lengths, 0).sum())
    assert 0 < T <= 2000
    run(lengths, *rest, T=T, block=4, in_place=in_place)
    run(lengths, *rest, T=2048, block=4, in_place=in_place, offset=1)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N", [8193, 16384])
@pytest.mark.parametrize("spare", [0, 1000])
def test_many_requests_that_do_not_fit(N, spare, in_place):
    b = books(N, 4, 8, 20, spare=spare, seed=spare, done=N // 20, lo=1, hi=9)
    total = int(np.maximum(b[0], 0).sum())
    assert run(*b, T=total, block=4, in_place=in_place)["cu"][-1] < total
    run(*b, T=total // 3, block=4, in_place=in_place)
    run(*b, T=1000, block=4, in_place=in_place)
    run(*b, T=0, block=4, in_place=in_place)


def test_bad_books_among_many_are_reported():
    lengths, ctx, *rest = books(16384, 4, 8, 16, spare=9000, seed=1, done=50, hi=2)
    lengths[[3, 9000, 16383]], ctx[[77, 12000]] = (-2, 10 ** 9, 40), (-1, 2 ** 31 - 1)
    T = int(np.clip(lengths, 0, 40).sum())
    run(lengths, ctx, *rest, T=T, block=4, in_place=True)
