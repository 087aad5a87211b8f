"""The compiled module of the plain calls where it is missing (no GPU needed): calls
go on without it and the first one says so, a build without it goes on and says so."""
import os
import sys
import warnings

import pytest
import torch

import __graft_entry__
import quantized_lora_fine_nf4_amd as q
from quantized_lora_fine_nf4_amd import build


@pytest.fixture
def no_module(monkeypatch):
    """As in an installation without _calls.so."""
    monkeypatch.setattr(q, "_plain", None)
    monkeypatch.delattr(q, "_calls", raising=False)
    monkeypatch.setitem(sys.modules, q.__name__ + "._calls", None)


def quantise():
    x, codes, scales = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    with pytest.raises(q.NF4Error, match="GPU"):   # Python's own checks
        q.mx4_quantize(x, codes, scales)


def test_the_first_call_without_it_says_so(no_module, recwarn):
    quantise()
    said = [w for w in recwarn if issubclass(w.category, RuntimeWarning)]
    assert len(said) == 1 and "small calls will be slower" in str(said[0].message)
    assert said[0].filename == __file__   # the caller's line
    quantise()
    assert len([w for w in recwarn if issubclass(w.category, RuntimeWarning)]) == 1


def test_warnings_as_errors_stop_the_first_call_alone(no_module):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeWarning):
            quantise()
        quantise()


def test_a_torch_without_the_raw_stream_says_so(monkeypatch):
    monkeypatch.setattr(q, "_plain", None)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    with pytest.warns(RuntimeWarning, match="small calls will be slower"):
        quantise()


def test_a_loaded_module_says_nothing(monkeypatch, recwarn):
    if not os.path.exists(build.CALLS_PATH) or not hasattr(torch._C, "_cuda_getCurrentRawStream"):
        pytest.skip("the module is not built, or this torch has no GPU part")
    monkeypatch.setattr(q, "_plain", None)
    quantise()
    assert not [w for w in recwarn if issubclass(w.category, RuntimeWarning)]


@pytest.mark.parametrize("why", ["compiler fails", "no compiler", "no torch"])
def test_a_build_goes_on_without_it(why, monkeypatch, tmp_path, capsys):
    path = tmp_path / "_calls.so"
    path.write_bytes(b"of an older source")
    monkeypatch.setattr(build, "CALLS_PATH", str(path))
    if why == "no torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr(build, "calls_command", lambda out: ["false" if why == "compiler fails" else str(tmp_path / "none")])
    assert build.build_calls_if_possible() is None
    assert not path.exists() and "was not built" in capsys.readouterr().err


def test_the_build_entry_point_goes_on_without_it(monkeypatch, tmp_path, capsys):
    """With every other part's build taken as done."""
    import oracle
    import synth
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "calls_command", lambda out: ["false"])
    for module, name in ((build, "build"), (build, "build_cpu"), (oracle, "build"), (synth, "build")):
        monkeypatch.setattr(module, name, lambda **kw: None)
    __graft_entry__.build()
    said = capsys.readouterr()
    assert "was not built" in said.err and "built" in said.out
