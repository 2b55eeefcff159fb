"""Shared helpers of the sequence-to-sequence operators' GPU tests."""
import numpy as np

# unit roundoff of a storage type, and the smallest step of its subnormals
UNIT = {"f32": 2.0**-24, "bf16": 2.0**-8, "f16": 2.0**-11}
TINY = {"f32": 2.0**-149, "bf16": 2.0**-133, "f16": 2.0**-24}
U32 = 2.0**-24


def code(lstm, dt):
    return {"f32": lstm.F32, "bf16": lstm.BF16, "f16": lstm.F16}[dt]


def tdtype(torch, dt):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt]


def stored(torch, a, dt):
    """numpy values -> (CPU tensor of the storage type, its values in fp64)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(tdtype(torch, dt))
    return t, t.double().numpy()


def host(t):
    return t.detach().cpu().double().numpy()


def within(got, want, tol, what=""):
    """|got - want| <= tol element by element; infinities and NaN in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = np.broadcast_to(tol, want.shape)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
    inf = np.isinf(want)
    np.testing.assert_array_equal(got[inf], want[inf], err_msg=what)
    fin = np.isfinite(want)
    assert np.isfinite(got[fin]).all(), f"{what}: not finite"
    d = np.abs(got[fin] - want[fin])
    worst = float((d / np.maximum(tol[fin], 1e-300)).max()) if d.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times the bound"
    return worst
