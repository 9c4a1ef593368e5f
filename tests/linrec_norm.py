"""The norm of the linear recurrence's errors, beside the bounds of single values in
tests/layer_ref.py: those grow with the length of a sequence and say little of an error that
all values share, such as that of a state carried in too few bits.

A value in fp32 is off by the errors of its terms.  A decay a = exp(-L) is off by 16 L + 5 steps of
2^-24 (tests/test_gpu_linrec.py), and a state adds up over about 1 / L tokens: the first part
comes to 16 steps whatever L is, the second, independent from token to token, to 5 / sqrt(L).
With decays of 0.999 a token and a gate that is nearly shut L is 0.004: 100 steps in all, and
some tens for the gates and the input.  The sums over tokens carry the same relative error as their
terms.  That is 8e-6 at the slowest channel; `near` asks for 1e-5.  Results in bf16 are
rounded once, which is at most half a step, 2^-8 of the value, spread evenly: 2^-8 / sqrt(3) in
norm if every value were at the lower end of its binade, where a step is largest."""
import torch

from tests.layer_ref import d

FP32 = 1e-5
BF16 = 2.0 ** -8 / 3 ** 0.5 + FP32


def near(got, ref, name):
    tol = FP32 if got.dtype == torch.float32 else BF16
    off, size = (d(got) - ref).norm().item(), ref.norm().item()
    assert off <= tol * size + 1e-30, f"{name}: the error's norm is {off / size:.3g} of the values', more than {tol:.3g}"
