"""What a handle's constructor sets stays set; other attributes are the user's."""

import pytest

from long_context_decode_c4a_b200.ops import _Handle


class Thing(_Handle):
    def __init__(self):
        self.a = 1
        self.a = 2      # until it is done
        self._fixed = frozenset(self.__dict__)


def test_fixed_attributes():
    t = Thing()
    t.note = "x"
    t.note = "y"
    del t.note
    for act in (lambda: setattr(t, "a", 3), lambda: delattr(t, "a")):
        with pytest.raises(AttributeError):
            act()
    assert t.a == 2 and not hasattr(t, "note")
