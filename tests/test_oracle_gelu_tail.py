"""The oracle's GELU far out in the negative tail, where Phi(z) = 1 + erf(z / sqrt 2) would cancel."""

import numpy as np
import pytest

import oracle as O


# Phi(-z), 13 digits of the published tables of the normal tail
@pytest.mark.parametrize("z,phi", [(1.0, 1.586552539315e-1), (3.0, 1.349898031630e-3), (6.0, 9.865876450377e-10),
                                   (8.0, 6.220960574272e-16), (10.0, 7.619853024161e-24)])
def test_gelu_keeps_its_relative_accuracy_in_the_tail(z, phi):
    # the table's last digit, and float64 rounding of the argument: z^2 steps of 2^-53
    assert abs(O.gelu_erf(np.array([-z]))[0] / (-z * phi) - 1.0) < 1e-12 + z * z * 2.0 ** -52
