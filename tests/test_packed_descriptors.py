"""The descriptors that the binding packs by itself have the layout of their C structures."""
import ctypes as C

import pytest

from invariant_forward_bitwise_gb300 import biv


@pytest.mark.parametrize("name,pack", [("LmLossDesc", "_pack_loss"), ("LmGradDesc", "_pack_grad"),
                                       ("NormFp8Desc", "_pack_norm"), ("NormBwdFp8Desc", "_pack_norm_bwd")])
def test_every_field_is_where_ctypes_has_it(name, pack):
    desc = getattr(biv, name)
    values = [float(i + 1) if kind is C.c_float else (1 << 40) + i if C.sizeof(kind) == 8 else i + 1
              for i, (_, kind) in enumerate(desc._fields_)]
    data = getattr(biv, pack)(*values)
    assert len(data) == C.sizeof(desc)
    back = desc.from_buffer_copy(data)
    assert [getattr(back, field) for field, _ in desc._fields_] == values
    assert all(getattr(desc.from_buffer_copy(getattr(biv, pack)(*[0] * len(values))), f) in (None, 0)
               for f, _ in desc._fields_)
