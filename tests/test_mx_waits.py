"""What a product reports when a wait inside its kernel runs out."""
import pytest
import torch

from tests.test_mx import BF, F32, check_product, quantised, ss  # noqa: F401

gpu = pytest.mark.gpu


def test_expired_wait_is_asked_for_with_a_truth_value(ss):  # noqa: F811
    for bad in (2, -1):
        with pytest.raises(ss.ShardStateError) as e:
            ss.ss_mx_expire_wait(bad)
        assert e.value.status == ss.SS_EINVAL
    ss.ss_mx_expire_wait(True)
    ss.ss_mx_expire_wait(False)


def unreached(M, N, sms):
    """Elements of out that the first CTA, or the first pair of them, would have made."""
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    m_tiles, n_tiles, pairs = -(-M // 256), -(-N // 256), sms // 2
    if 2 * m_tiles * n_tiles >= pairs and M > 128 and N > 128:
        for t in range(0, m_tiles * n_tiles, pairs):
            m, n = t % m_tiles * 256, t // m_tiles * 256
            bad[m:m + 256, n:n + 256] = True
    else:
        swap = N < M and N <= 128
        few = N if swap else M
        few = 16 if few <= 16 else 32 if few <= 32 else 64 if few <= 64 else 128
        (bad.t() if not swap else bad)[:128, :few] = True
    return bad


@gpu
@pytest.mark.parametrize("M,N,K,format,dtype", [
    (1, 300, 5632, 0, BF), (40, 1100, 200, 1, F32), (1021, 70, 1001, 0, BF), (300, 200, 130, 1, BF),
    (2500, 2600, 300, 0, BF), (2048, 5632, 520, 1, F32)])
def test_a_wait_that_runs_out(ss, M, N, K, format, dtype):  # noqa: F811
    """One wait that nothing ends gives up by itself: its tiles are NaN, the others right, and so is the next call."""
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    (qa, a), (qb, b) = quantised(ss, M, K, format, gen), quantised(ss, N, K, format, gen)
    out, good = (torch.full((M, N), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    ss.ss_mx_expire_wait(True)
    ss.ss_mx_matmul(*qa, *qb, K, format, torch.empty(0, N, device="cuda"))  # launches nothing
    ss.ss_mx_matmul(*qa, *qb, K, format, out)
    ss.ss_mx_matmul(*qa, *qb, K, format, good)
    check_product(good, a, b)
    bad = unreached(M, N, torch.cuda.get_device_properties(0).multi_processor_count)
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], good[~bad])
