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
