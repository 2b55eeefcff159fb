"""The fp64 reference of linear attention, penalties and AdamW against brute
force, central differences and the number format's own table (no GPU)."""
import numpy as np
import pytest

from oracle import model_oracle as mo


def case(seed=0, T=6, B=3, Hq=4, Hk=2, D=5, Dv=3):
    r = np.random.default_rng(seed)
    n = r.normal
    return dict(q=n(size=(T, B, Hq, D)), k=n(size=(T, B, Hk, D)), v=n(size=(T, B, Hk, Dv)),
                log_decay=np.array([-0.3, 0.4]), scale=0.7, state=n(size=(B, Hk, D, Dv)), length=np.array([6, 0, 4]),
                do=n(size=(T, B, Hq, Dv)), dstate=n(size=(B, Hk, D, Dv)))


def test_linear_attention_is_the_sum_over_the_steps_before():
    c = case()
    o, S = mo.linattn(c["q"], c["k"], c["v"], c["log_decay"], c["scale"], c["state"], c["length"])
    T, B, Hq, _ = c["q"].shape
    for b in range(B):
        for h in range(Hq):
            a, hk = np.exp(min(c["log_decay"][h // 2], 0)), h // 2
            for t in range(T):
                want = 0.0
                if t < c["length"][b]:
                    want = a ** (t + 1) * c["q"][t, b, h] @ c["state"][b, hk]
                    for j in range(t + 1):
                        want = want + a ** (t - j) * (c["q"][t, b, h] @ c["k"][j, b, hk]) * c["v"][j, b, hk]
                np.testing.assert_allclose(o[t, b, h], c["scale"] * want, atol=1e-12)
    np.testing.assert_array_equal(S[1], c["state"][1])


def test_linear_attention_gradients_by_differences():
    c = case(1)

    def loss(**new):
        d = dict(c, **new)
        o, S = mo.linattn(d["q"], d["k"], d["v"], d["log_decay"], d["scale"], d["state"], d["length"])
        return (o * c["do"]).sum() + (S * c["dstate"]).sum()

    grads = mo.linattn(**c)[2:]
    r = np.random.default_rng(2)
    for name, g in zip(("q", "k", "v", "state"), grads):
        d = r.normal(size=g.shape)
        slope = (loss(**{name: c[name] + 0.5 * d}) - loss(**{name: c[name] - 0.5 * d}))  # linear in each argument
        assert abs(slope - (g * d).sum()) < 1e-9 * max(1, abs(slope)), name


def test_penalties_by_hand():
    x = np.array([[2.0, -1.0, 0.5, 3.0]])
    y = mo.penalty(x, np.array([[0, 1, 1, -1, 9, 3]]), np.array([5]), np.array([2.0]), np.array([0.25]), np.array([0.5]),
                   np.array([0.0, 0.0, 1.0, 0.0]), np.array([[True, True, True, False]]))
    np.testing.assert_array_equal(y, [[2 / 2 - 0.25 - 0.5, -2 - 0.25 - 1.0, 1.5, -np.inf]])


def test_adamw_against_torch():
    torch = pytest.importorskip("torch")
    p = torch.randn(50, dtype=torch.float64, requires_grad=True)
    w, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    for t in range(1, 4):
        p.grad = torch.randn(50, dtype=torch.float64)
        w, m, v = mo.adamw(w, p.grad.numpy(), m, v, t, 0.01, 0.9, 0.99, 1e-8, 0.1)
        opt.step()
        np.testing.assert_allclose(w, p.detach().numpy(), rtol=1e-12)


def test_e4m3_numbers():
    torch = pytest.importorskip("torch")
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.sort(codes), mo.e4m3_values())
    x = np.linspace(0, 440, 100001)
    near = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert (np.abs(near - x) <= mo.e4m3_step(x) / 2).all()
