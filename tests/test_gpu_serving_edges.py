"""The serving operators where it is easy to go wrong: values that are not finite or very large
beside keys that a row does not see, scales far apart, freed pages, status and streams.  References
and tolerances as in test_gpu_serving.py."""
import numpy as np
import pytest

import tiled_tensor_core_03_gb300 as gr

import serving_reference as ref
from test_gpu_serving import DTYPES, _cache, _check, _cuda, _dt, _f64, _half_step, _i32, _rand, _tables  # noqa: F401

pytestmark = pytest.mark.gpu

# ---------------------------------------------------------------- flash_attention_window


def _sees(n, at, window, sinks):
    return np.array([at <= p and (window == 0 or at > p - window or at < sinks) for p in range(n)])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [2, 64, 130])
def test_window_not_finite_beside_rows_that_left_sinks_behind(sinks, d, dtype):
    """Rows whose window has left some of the sinks behind (positions from window to window + sinks)
    beside a V that is not finite, in a key they do not see and in a sink: every element that it
    does not reach is as the formula says, also in the rows that see it."""
    rng = np.random.default_rng(sinks + d)
    n, window = 300, 40
    q, q64 = _rand(rng, (1, n, 2, d), dtype)
    k, k64 = _rand(rng, (1, n, 1, d), dtype)
    v, v64 = _rand(rng, (1, n, 1, d), dtype)
    for at, value in ((window + min(sinks, 80) + 1, np.nan), (120, np.inf), (1, np.inf), (299, -np.inf)):
        vv, vv64 = v.clone(), v64.copy()
        vv[0, at, 0, 5] = value
        vv64[0, at, 0, 5] = value
        got = _f64(gr.flash_attention_window(q, k, vv, window, sinks))[0]
        o, absv, _, size = ref.attend(q64[0], k64[0], vv64[0], window, sinks)
        sees = _sees(n, at, window, sinks)
        assert not np.isfinite(got[sees][..., 5]).any()
        _check(got[~sees], o[~sees], absv[~sees], size[~sees], d, dtype, _half_step(dtype))
        got, o, absv = (np.delete(x, 5, 2) for x in (got, o, absv))
        _check(got, o, absv, size, d, dtype, _half_step(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_window_first_score_minus_infinity(dtype):
    """A key whose score is -infinity has weight 0, also where it is the first that a row sees and
    a V that the row does not see is not finite."""
    rng = np.random.default_rng(41)
    n, d = 200, 64
    q, q64 = _rand(rng, (1, n, 1, d), dtype)
    k, k64 = _rand(rng, (1, n, 1, d), dtype)
    v, v64 = _rand(rng, (1, n, 1, d), dtype)
    q, q64 = q.abs(), np.abs(q64)
    k[0, :2, 0, 5], k64[0, :2, 0, 5] = -np.inf, -np.inf
    v[0, 199, 0, 7], v64[0, 199, 0, 7] = np.nan, np.nan
    for window, sinks in ((0, 0), (50, 2)):
        got = _f64(gr.flash_attention_window(q, k, v, window, sinks))[0, 2:199]
        with np.errstate(invalid="ignore"):
            o, absv, _, _ = ref.attend(q64[0], k64[0], v64[0], window, sinks)
        size = ref.attend(q64[0], np.where(np.isinf(k64[0]), 0, k64[0]), v64[0], window, sinks)[3]
        _check(got, o[2:199], absv[2:199], size[2:199], d, dtype, _half_step(dtype))
