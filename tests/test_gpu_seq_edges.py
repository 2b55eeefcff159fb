"""The sequence-to-sequence operators at the edges of what they take: tensors
elsewhere than on the device, rows that overlap, other streams, probabilities
and gradients at the ends of a type's range, rows of NaN, sizes at the launch
limits.  References are fp64 (oracle/seq_oracle.py) or the definition."""
import numpy as np
import pytest

from oracle import seq_oracle as so
from seq_util import TINY, U32, UNIT, code, host, stored, tdtype, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def test_each_tensor_has_to_be_on_the_device(lstm):
    """Every argument in turn left in host memory: refused before any launch."""
    cu = lambda *a: torch.ones(*a, device="cuda")  # noqa: E731
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    e = lstm.Embedding(4, 9, 8)
    a = lstm.Attention(2, 3, 2, 2, 1, 8)
    q, k, n, mask = cu(2, 2, 2, 8), cu(3, 2, 1, 8), torch.full((2,), 3, dtype=torch.int32, device="cuda"), cu(2, 3).bool()
    p = lstm.LogProb(4, 9, top=2)
    p.forward(cu(4, 9), ids)
    for f, args in ((e.forward, (ids, cu(9, 8))), (e.backward, (ids, cu(4, 8))), (a.forward, (q, k, k, n, mask)),
                    (a.backward, (q, q, k, k, n, mask)), (p.forward, (cu(4, 9), ids)),
                    (p.backward, (cu(4, 9), ids, cu(4), cu(4), cu(4, 2)))):
        f(*args)
        for i in range(len(args)):
            with pytest.raises(ValueError, match="cuda:0"):
                f(*(x.cpu() if j == i else x for j, x in enumerate(args)))
    torch.cuda.synchronize()


def test_outputs_made_for_another_stream(lstm):
    """The current stream still has a fill of a freed tensor ahead of it; an
    output first made for a call on another stream is not that memory."""
    N, V, D, busy = 64, 20000, 1024, 400_000_000  # clock cycles, about 0.2 s
    s = torch.cuda.Stream()
    ids, dout = torch.zeros(N, dtype=torch.int64, device="cuda"), torch.ones(N, D, device="cuda")
    x, g = torch.randn(N, V, device="cuda"), torch.ones(N, device="cuda")
    q, k = torch.randn(512, 8, 16, 64, device="cuda"), torch.randn(512, 8, 16, 64, device="cuda")
    e, p, a = lstm.Embedding(N, V, D), lstm.LogProb(N, V, top=2), lstm.Attention(512, 512, 8, 16, 16, 64)
    p.forward(x, ids), a.forward(q, k, k)
    e2, p2, a2 = lstm.Embedding(N, V, D), lstm.LogProb(N, V, top=2), lstm.Attention(512, 512, 8, 16, 16, 64)
    p2.forward(x, ids), a2.forward(q, k, k)
    calls = [(V * D, lambda m, st: m.backward(ids, dout, stream=st), e, e2),
             (N * V, lambda m, st: m.backward(x, ids, g, stream=st), p, p2),
             (q.numel(), lambda m, st: m.backward(q, q, k, k, stream=st), a, a2)]
    for n, call, other, own in calls:
        want = call(own, None)
        want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
        torch.cuda.synchronize()
        freed = [torch.empty(n, device="cuda") for _ in want]
        torch.cuda._sleep(busy)
        for t in freed:
            t.fill_(7.0)
        del freed, t
        got = call(other, s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got if isinstance(got, tuple) else (got,), want))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_alternatives_of_short_rows_are_all_there(lstm, dt):
    """Rows of a few logits, banned ones among them, as many alternatives as logits, at every offset from 16 bytes: each
    id once, ties by the lower."""
    rng = np.random.default_rng(2)
    for V in (1, 2, 3, 5, 6, 7, 9, 13, 18, 21, 27, 31):
        x = rng.normal(size=(17, V))  # 17 rows of V: at most offsets
        x[rng.random(x.shape) < 0.4] = -np.inf
        x[3] = -np.inf
        xs, x64 = stored(torch, x, dt)
        m = lstm.LogProb(17, V, code(lstm, dt), top=V)
        ids = m.forward(xs.cuda(), torch.zeros(17, dtype=torch.int64, device="cuda"))[3].cpu().numpy()
        np.testing.assert_array_equal(ids, so.logprob(x64, np.zeros(17), 1.0, V)["top_ids"], err_msg=f"V = {V}")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [5, 300, 70000])
def test_ids_of_rows_with_nan_are_tokens(lstm, dt, V):
    """NaN of either sign, a few, among banned tokens, or nothing else: the alternatives are NaN first, then the largest,
    and every id is one of the row's, once."""
    rng = np.random.default_rng(3)
    x, _ = stored(torch, rng.normal(size=(8, V)), dt)
    nan = torch.tensor([0x7FC00000, -0x400000], dtype=torch.int32).view(torch.float32).to(x.dtype)
    x[0], x[1] = nan[0], nan[1]
    x[2], x[3] = -np.inf, -np.inf
    x[2, V // 2], x[3, V // 2] = nan[0], nan[1]
    x[4, 1::2], x[5, 1::2] = nan[0], nan[1]
    x[6, V - 1] = nan[1]
    top = 4
    m = lstm.LogProb(8, V, code(lstm, dt), top=top)
    ids = m.forward(x.cuda(), torch.zeros(8, dtype=torch.int64, device="cuda"))[3]
    h = x.double().numpy()
    want = np.argsort(-np.where(np.isnan(h), np.inf, h), axis=1, kind="stable")[:, :top]
    np.testing.assert_array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_nan_far_along_a_row_of_numbers(lstm, dt):
    """Each row a NaN at another place, among logits that rank high and low, in one and in several parts."""
    g = torch.Generator(device="cuda").manual_seed(2)
    for N, V in ((2300, 20011), (40, 20011)):
        x = torch.randn(N, V, generator=g, device="cuda")
        x[:, 7] = 50.0
        at = torch.randint(8, V, (N,), generator=g, device="cuda")
        x[torch.arange(N, device="cuda"), at] = float("nan")
        m = lstm.LogProb(N, V, code(lstm, dt), top=2)
        ids = m.forward(x.to(tdtype(torch, dt)), torch.zeros(N, dtype=torch.int64, device="cuda"))[3]
        assert torch.equal(ids, torch.stack([at, torch.full_like(at, 7)], 1))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [5, 300, 70000])
def test_nan_in_a_row_without_numbers(lstm, dt, V):
    """A row of NaN, one of banned tokens and a NaN: every sum and gradient of it is NaN, its neighbours' are not."""
    x = torch.zeros(4, V, dtype=tdtype(torch, dt), device="cuda")
    x[0], x[1], x[3] = float("nan"), float("-inf"), float("-inf")
    x[1, V - 1] = float("nan")
    t = torch.tensor([0, 1, 2, 3], device="cuda")
    one = torch.ones(4, device="cuda")
    m = lstm.LogProb(4, V, code(lstm, dt), top=2)
    logp, H, tl, _ = m.forward(x, t)
    g = m.backward(x, t, one, one)
    for a in (logp, m.lse, H, tl, g):
        assert torch.isnan(a[:2]).all() and not torch.isnan(a[2:]).any()
    assert torch.isneginf(logp[3]) and torch.isneginf(m.lse[3]) and H[3] == 0 and not g[3].any()


def test_attention_without_heads(lstm):
    m = lstm.Attention(3, 4, 2, 0, 0, 16)
    q, k = torch.empty(3, 2, 0, 16, device="cuda"), torch.empty(4, 2, 0, 16, device="cuda")
    o, lse = m.forward(q, k, k)
    grads = m.backward(q, q, k, k)
    torch.cuda.synchronize()
    assert o.shape == (3, 2, 0, 16) and lse.shape == (2, 0, 3) and [g.shape for g in grads] == [q.shape, k.shape, k.shape]


def test_embedding_of_the_most_tokens_and_rows(lstm):
    """One less than 2^26 of each: more rows than one launch of a wave each has threads for."""
    n = (1 << 26) - 1
    torch.cuda.empty_cache()
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-1, 10, (n,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.randn(10, 2, generator=g, device="cuda").half()
    out = lstm.Embedding(n, 10, 2, lstm.F16).forward(ids, table)
    for lo in (0, n // 2, n - 1000):
        part = ids[lo : lo + 1000].long()
        want = torch.where((part >= 0)[:, None], table[part.clamp(min=0)], 0.0)
        assert torch.equal(out[lo : lo + 1000], want.half())
    del out
    ids, dout = torch.tensor([0, n - 1, n - 2, n // 2, n - 1], device="cuda"), torch.randn(5, 2, generator=g, device="cuda").half()
    m = lstm.Embedding(5, n, 2, lstm.F16)
    m.dtable = torch.full((n, 2), float("nan"), dtype=torch.float16, device="cuda")
    got = m.backward(ids, dout)
    assert torch.equal(got[[0, n - 2, n // 2]], dout[[0, 2, 3]]) and (got != 0).any(1).sum() == 4
    assert torch.equal(got[n - 1], (dout[1].float() + dout[4].float()).half())


def test_gradient_of_the_most_rows(lstm):
    """2^23 rows of 4097 logits, 137 GB, in place: more work-groups than one launch has threads for.  All rows but
    a few are equal logits with no cotangent."""
    N, V = 1 << 23, 4097
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160e9:
        pytest.skip("needs 160 GB of free device memory")
    x = torch.zeros(N, V, device="cuda")
    # one launch has 2^24 - 1 work-groups, two of them a row: the first starts again at row 2^23 - 1
    rows = [0, 12345, N // 2, N - 3, N - 2, N - 1]
    rng = np.random.default_rng(5)
    part, part64 = stored(torch, rng.normal(size=(len(rows), V)), "f32")
    x[rows] = part.cuda()
    t = torch.full((N,), -1, device="cuda")
    dl, dh = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    tr, lr, hr = rng.integers(0, V, len(rows)), rng.normal(size=len(rows)), rng.normal(size=len(rows))
    t[rows], dl[rows], dh[rows] = (torch.from_numpy(a).to(b.dtype).cuda() for a, b in ((tr, t), (lr, dl), (hr, dh)))
    m = lstm.LogProb(N, V, lstm.F32)
    m.forward(x, t)
    m.dlogits = x
    m.backward(x, t, dl, dh)
    got = host(x[rows])
    want = so.logprob(part64, tr, 1.0, 0, lr.astype(np.float32), hr.astype(np.float32))["dlogits"]
    within(got, want, 2e-5 * np.abs(want) + 1e-9, "dlogits")
    mid = [1, N // 3, N - 4]
    assert not x[mid].any()
    del x, m
    torch.cuda.empty_cache()
