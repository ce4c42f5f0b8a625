"""The package has a function of the name of every C entry point that takes a
stream, whichever module it stands in."""
import inspect

import pytest

import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import api, experts, feedforward


def test_every_call_is_found_in_the_package():
    from group_scaling_fp8_amd import mgs_mm_gated_i8
    assert mgs_mm_gated_i8 is feedforward.mgs_mm_gated_i8
    for module in (api, experts, feedforward):
        for name, f in vars(module).items():
            if name.startswith("mgs_") and inspect.isfunction(f):
                assert getattr(mgs, name) is f and name in dir(mgs), name


def test_other_names_are_not():
    assert not hasattr(mgs, "mgs_mm_i4")
    with pytest.raises(AttributeError, match="mgs_mm_i4"):
        mgs.mgs_mm_i4
