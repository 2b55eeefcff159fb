"""Penalties on so many rows that one launch has not enough work-groups for them
(one of 512 threads a row, fewer than 2^32 threads a launch: 2^23 - 1 rows): the
rows on both sides of the place where a launch ends, and all others, by the same
fp32 operations in torch."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


@pytest.mark.parametrize("counts", [True, False])
def test_rows_of_two_launches(lstm, counts):
    N, V = (1 << 23) + 1000, 3
    print(f"case: penalty, {N} rows of {V} logits, history {counts}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((N, V), generator=g, device="cuda").bfloat16()
    mask = torch.randint(0, 8, (N, 1), generator=g, device="cuda", dtype=torch.int32)
    bias = torch.randn(V, generator=g, device="cuda")
    m = lstm.Penalty(N, V, lstm.BF16)
    m.out = torch.full((N, V), 7.0, dtype=torch.bfloat16, device="cuda")
    want, how = x.float(), {}
    if counts:
        # one token said by each row (3: nobody's), its penalty a whole number
        said = torch.randint(0, V + 1, (N, 1), generator=g, device="cuda", dtype=torch.int32)
        presence = torch.randint(1, 9, (N,), generator=g, device="cuda").float()
        want = want - torch.where(said == torch.arange(V, device="cuda"), presence[:, None], 0.0)
        how = dict(history=said, presence=presence)
    want = want + bias
    want = torch.where((mask >> torch.arange(V, device="cuda", dtype=torch.int32)) & 1 != 0, want, float("-inf")).bfloat16()
    got = m.forward(x, bias=bias, mask=mask, **how)
    torch.cuda.synchronize()
    for lo, hi in ((0, 2), ((1 << 23) - 3, (1 << 23) + 3), (N - 2, N), (0, N)):
        assert torch.equal(got[lo:hi], want[lo:hi]), (lo, hi)
