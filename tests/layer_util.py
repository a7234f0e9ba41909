"""Helpers of the tests of the operators around the scan."""
import numpy as np

from mamba_ssd_scan_chunked_b200 import inputs as I
from tests.gpu_util import bf16_excess_metric, metric, to_dev, to_host64, torch

# max|err| / rms(oracle) of an fp32 result; a bf16 result may be off by half a
# bf16 step of the value on top of it (its one rounding, 2^-8 of the value at most).
#
# Arithmetic: inputs are exact on both sides and every kernel computes in fp32
# from them.  An output is a sum of at most n products, each formed with k
# roundings of 2^-24 and the approximations of exp, log, division and square
# root (2 to 4 units of 2^-23 each, so k <= 40 in units of 2^-24 counts a chain
# of four of them and their arguments).  A carried state adds one such chain per
# token, damped by the decays, and the sums behind a gradient one rounding per
# term: errors of independent sign, whose size grows as the square root of the
# count.  With n <= 4000 terms in the tests, sqrt(4000) * 2^-24 * 40 = 1.5e-4 of
# a single term's size, and the sum's rms is sqrt(n) of it: below 1e-5 of the
# rms for the typical element, and the largest of 10^6 elements (5 sigma) below
# 5e-5.  1e-4 is the method's own bound for fp32.
TOL = 1e-4


def draw(seed, shape, dtype, std=1.0, loc=0.0):
    """A normal storage array (fp32, or bf16 bits)."""
    return I.to_storage(np.random.default_rng(seed).normal(loc, std, shape), dtype)


def t_dtype(name):
    return torch().bfloat16 if name == I.BF16 else torch().float32


def check(name, got, ref):
    if ref is None:
        assert got is None, name
        return
    assert tuple(got.shape) == ref.shape, (name, got.shape, ref.shape)
    host = to_host64(got)
    assert np.isfinite(host).all(), name
    if not ref.size:
        return
    if not ref.any():
        assert not host.any(), name
        return
    err = (bf16_excess_metric if got.dtype == torch().bfloat16 else metric)(host, ref)
    assert err <= TOL, (name, err)


def check_dict(got, ref):
    assert set(got) == set(ref)
    for k in ref:
        check(k, got[k], ref[k])


def rows_of(a, extra, fill=float("nan")):
    """The array as the last columns of wider rows (`extra` more elements, filled with `fill`)."""
    t = torch()
    dense = to_dev(a)
    wide = t.full(dense.shape[:-1] + (dense.shape[-1] + extra,), fill, dtype=dense.dtype, device="cuda")
    wide[..., extra:] = dense
    return wide[..., extra:]


def dev(a):
    return None if a is None else to_dev(a)


def f64(a):
    return None if a is None else I.to_f64(a)
