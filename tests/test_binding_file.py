"""The extension of the operators' plain calls holds the layouts of the interpreter and the torch that
it was built for: one of others is not loaded."""
import os
import sysconfig

import pytest


def test_the_file_in_use_is_the_one_for_this_interpreter_and_torch():
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint
    from newton_schulz_13_b200 import build, gradients
    assert gradients._fast is not None
    assert os.path.samefile(gradients._fast.__file__, build.binding_path())
    assert not build.binding_stale()


@pytest.mark.parametrize("what", ["torch", "commit", "interpreter"])
def test_a_file_built_for_others_is_stale(what, monkeypatch):
    import torch

    from newton_schulz_13_b200 import build
    build.build_binding()
    assert not build.binding_stale()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif what == "commit":
        monkeypatch.setattr(torch.version, "git_version", "0123456789abcdef")
    else:
        var = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-00-none" if n == "SOABI" else var(n))
    assert build.binding_stale()
