"""When the binding's marshalling is compiled again (host only: the compiler is a stand-in)."""
import shutil
import sysconfig

import pytest
import torch


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """(build module on a copy of the built binding, commands it has run)."""
    import __graft_entry__
    __graft_entry__.build()
    from bit_quantized_gemm_quant_b200 import build as b
    commands = []

    def compiler(cmd):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()

    monkeypatch.setattr(b, "BINDING", shutil.copy2(b.BINDING, str(tmp_path)))
    monkeypatch.setattr(b.subprocess, "check_call", compiler)
    b.build()
    commands.clear()
    return b, commands


def test_binding_is_kept_while_nothing_changes(compiled):
    b, commands = compiled
    b.build()
    assert commands == []


@pytest.mark.parametrize("change", ["torch", "python"])
def test_binding_follows_pytorch_and_python(compiled, monkeypatch, change):
    b, commands = compiled
    with monkeypatch.context() as m:
        if change == "torch":
            m.setattr(torch, "__version__", torch.__version__ + ".other")
        else:
            m.setattr(sysconfig, "get_config_var", lambda name: "cpython-other")
        for _ in range(2):
            b.build()
        assert len(commands) == 1 and "-shared" in commands[0]
    b.build()
    assert len(commands) == 2
