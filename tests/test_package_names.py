"""The package's names are its modules' own.  CPU only."""

import pytest

import lm_output_head_amd


@pytest.mark.parametrize("module,name", [("serve", "rmsnorm"), ("serve", "fh_w8a8_matmul"), ("fp8", "fp8_quant"),
                                         ("beam", "beam_select"), ("flashhead", "fh_forward")])
def test_what_replaces_a_modules_name_is_the_packages(monkeypatch, module, name):
    """Before the name was used through the package, and after."""
    held = __import__("lm_output_head_amd." + module, fromlist=[name])
    real = getattr(held, name)
    assert getattr(lm_output_head_amd, name) is real
    with monkeypatch.context() as m:
        m.setattr(held, name, lambda *a, **k: None)
        assert getattr(lm_output_head_amd, name) is getattr(held, name) is not real
    assert getattr(lm_output_head_amd, name) is real


def test_unknown_names():
    with pytest.raises(AttributeError):
        lm_output_head_amd.no_such_name
