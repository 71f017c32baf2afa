"""What the tensor functions of the operators around the recurrence see to on the host: checks before any GPU work,
the device of a call, and the library's loading (CPU only)."""

import os
import subprocess
import sys

import pytest
import torch

from hybrid_linear_attention_prefill_gb300 import build as B
from hybrid_linear_attention_prefill_gb300 import gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return gdn.load()


class Entries:
    """Stands in for the library: notes the calls of its entries and returns 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append(name)
            return 0
        return entry


@pytest.fixture
def entries(monkeypatch):
    e = Entries()
    monkeypatch.setattr(gdn, "load", lambda *a: e)
    monkeypatch.setattr(gdn, "_fast", None)
    monkeypatch.setattr(gdn, "_raw_stream", lambda *a: 0)
    return e


def scan_operands(n=8):
    z, bf = torch.zeros, torch.bfloat16
    return dict(x=z(n, 4, 64, dtype=bf), dt=z(n, 4), A=z(4), Bm=z(n, 2, 32, dtype=bf), Cm=z(n, 2, 32, dtype=bf))


@pytest.mark.parametrize("workspace", [
    torch.zeros(4096, dtype=torch.uint8)[::2],          # strided: its bytes are not in one piece
    torch.zeros(64, 64, dtype=torch.uint8).t(),
    torch.zeros(4096, dtype=torch.uint8, device="meta")])  # on another device than x
def test_scan_refuses_a_workspace_that_is_not_one_piece_beside_x(entries, workspace):
    with pytest.raises(ValueError, match="workspace"):
        gdn.ssm_scan(**scan_operands(), workspace=workspace)
    assert entries.calls == []
    gdn.ssm_scan(**scan_operands(), workspace=torch.zeros(4096, dtype=torch.uint8))
    assert entries.calls == ["gdn_ssm_scan"]


# ---- the device of a call -----------------------------------------------------------------------

class OnDevice1(torch.Tensor):
    def get_device(self):
        return 1


def calls_on_device_1():
    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice1)

    f32 = torch.float32
    s = dict(x=t(8, 4, 64), dt=t(8, 4, dtype=f32), A=t(4, dtype=f32), Bm=t(8, 2, 32), Cm=t(8, 2, 32))
    return [("gdn_conv", lambda: gdn.causal_conv(t(8, 64), t(64, 4), out=t(8, 64), want_final=False)),
            ("gdn_conv_step", lambda: gdn.causal_conv_step(t(8, 64), t(64, 4), t(8, 3, 64), out=t(8, 64))),
            ("gdn_ssm_scan", lambda: gdn.ssm_scan(**s, out=t(8, 4, 64), want_final=False)),
            ("gdn_ssm_step", lambda: gdn.ssm_step(**s, state=t(8, 4, 64, 32, dtype=f32), out=t(8, 4, 64))),
            ("gdn_add_norm", lambda: gdn.add_norm(t(8, 64), t(64), out=t(8, 64)))]


@pytest.mark.parametrize("which", range(5))
def test_calls_run_with_the_device_of_x_as_the_current_one(monkeypatch, which):
    """The C entries launch on the current device, so it has to be the one that the operands and the stream are of."""
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.was

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, current[0])) or 0

    monkeypatch.setattr(gdn, "load", lambda *a: Lib())
    monkeypatch.setattr(gdn, "_fast", None)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    name, call = calls_on_device_1()[which]
    call()
    assert seen == [(name, 1)] and current == [0]


def test_a_stream_of_another_device_is_refused():
    class Stream:
        cuda_stream = 5
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream"):
        gdn._raw_stream(Stream(), 0)
    assert gdn._raw_stream(Stream(), 1) == 5 and gdn._raw_stream(7, 0) == 7


# ---- loading ------------------------------------------------------------------------------------

def run_python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_the_library_loads_without_pytorch():
    r = run_python("import sys; sys.modules['torch'] = None\n"
                   "from hybrid_linear_attention_prefill_gb300 import gdn\n"
                   "gdn.load(); print(gdn.gdn_abi_version(), gdn.gdn_prefill(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 1, 32, "
                   "32, 0))")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [str(gdn.gdn_abi_version()), "0"]


def test_loading_the_library_does_not_import_pytorch():
    r = run_python("import sys\nfrom hybrid_linear_attention_prefill_gb300 import gdn\n"
                   "gdn.load(); print('torch' in sys.modules)")
    assert r.returncode == 0 and r.stdout.split() == ["False"], r.stderr


@pytest.mark.parametrize("content", [b"", b"no shared object"])
def test_the_tensor_functions_do_without_a_module_that_does_not_load(tmp_path, content):
    bad = tmp_path / "gdn_torch.so"
    bad.write_bytes(content)
    r = run_python("import torch\nfrom hybrid_linear_attention_prefill_gb300 import build, gdn\n"
                   f"build.TORCH_LIB = {str(bad)!r}\nbuild.torch_lib = lambda: {str(bad)!r}\n"
                   "gdn.load(); z = torch.zeros\n"
                   "try: gdn.add_norm(z(2, 8).bfloat16(), z(8).bfloat16(), out=z(2, 8).bfloat16())\n"
                   "except ValueError as e: print(e)")
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "CUDA tensors are wanted"  # what the checks in Python say to host tensors


def test_the_module_is_of_this_interpreter_and_this_pytorch(monkeypatch):
    """Built against another PyTorch it could load and read its objects wrongly: its name says what it is for."""
    path = B.torch_lib()
    assert os.path.exists(path) and not B.module_needs_build()
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    assert B.torch_lib() != path and B.module_needs_build() and not B.needs_build()
    monkeypatch.setattr(gdn, "_fast", gdn._UNTRIED)
    assert gdn._shorter() is None  # there is none for that PyTorch


def test_only_the_module_is_built_for_another_pytorch(monkeypatch, tmp_path):
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        if "-o" in cmd:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B, "torch_lib", lambda: str(tmp_path / "gdn_torch.other.so"))
    monkeypatch.setattr(subprocess, "run", run)
    was = os.path.getmtime(B.LIB)
    B.build()
    assert [os.path.basename(c[0]) for c in calls] == ["g++", "g++"] and os.path.getmtime(B.LIB) == was
    B.build()
    assert len(calls) == 2  # it is there


def test_a_module_that_does_not_build_is_not_tried_at_every_call(monkeypatch, tmp_path, capsys):
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "no headers")

    path = tmp_path / "gdn_torch.other.so"
    path.touch()
    os.utime(path, (0, 0))  # older than its source
    monkeypatch.setattr(B, "torch_lib", lambda: str(path))
    monkeypatch.setattr(subprocess, "run", run)
    B.build()
    B.build()
    assert len(calls) == 1 and not path.exists() and "check in Python" in capsys.readouterr().out


# ---- ranges -------------------------------------------------------------------------------------

def test_sizes_beyond_32_bits_are_refused(entries):
    bf, z = torch.bfloat16, torch.zeros
    many = z(1, 64, dtype=bf).expand(2 ** 31, 64)
    x, w, st = z(8, 64, dtype=bf), z(64, 4, dtype=bf), z(8, 3, 64, dtype=bf)
    none = z(0, 64, dtype=bf)
    for call in (lambda: gdn.causal_conv(many, w), lambda: gdn.causal_conv_step(many, w, st),
                 lambda: gdn.add_norm(many, w[:, 0]), lambda: gdn.causal_conv(none, w, B=2 ** 31),
                 lambda: gdn.causal_conv(x, w, B=2 ** 70), lambda: gdn.add_norm(x, z(64, dtype=bf), group=2 ** 31),
                 lambda: gdn.add_norm(x, z(64, dtype=bf), e4m3=True, group=-1),
                 lambda: gdn.ssm_scan(**{**scan_operands(), "x": z(1, 4, 64, dtype=bf).expand(2 ** 31, 4, 64)})):
        with pytest.raises(ValueError):
            call()
    assert entries.calls == []
