"""gqa_tree_attn without a mask, or without cached lengths, is refused by name (CPU only)."""
import pytest

from test_binding_devices import native as binding  # noqa: F401  (the fixture)
from test_binding_devices_pages import arguments, native  # noqa: F401


@pytest.mark.parametrize("which", ["tree_mask", "cached_lens"])
def test_what_a_tree_needs(native, which):  # noqa: F811
    with pytest.raises(ValueError, match=which):
        native.gqa_tree_attn(**dict(arguments("gqa_tree_attn"), **{which: None}))
    assert native.lib.calls == 0
