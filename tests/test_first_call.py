"""Every entry point goes through torch's initialisation of CUDA, which starts it where nothing has yet and refuses a
process forked after it."""
import os

import pytest
import torch

import sparse_attention_06_b200 as dsa


class Asked(Exception):
    pass


@pytest.fixture
def lazy_init(monkeypatch):
    def asked():
        raise Asked
    monkeypatch.setattr(torch.cuda, "_lazy_init", asked)


def test_the_current_stream_asks_for_cuda_to_be_initialised(lazy_init):
    with pytest.raises(Asked):
        dsa._stream(None)


def test_calls_that_compare_devices_ask_too(lazy_init):
    with pytest.raises(Asked):
        dsa._same_device()


def test_a_given_stream_is_taken_as_it_is(lazy_init):
    assert dsa._stream(5) == 5


FIRST = """
import sparse_attention_06_b200 as dsa
dsa.dsa_clear_device_error()
print(dsa.dsa_get_device_error())
"""

FORKED = """
import os, torch
import sparse_attention_06_b200 as dsa
torch.cuda.init()
pid = os.fork()
if pid == 0:
    try:
        dsa.dsa_clear_device_error()
    except RuntimeError as e:
        os._exit(0 if "fork" in str(e) else 3)
    os._exit(4)
print(os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]))
"""


@pytest.mark.gpu
@pytest.mark.parametrize("program", [FIRST, FORKED], ids=["first", "forked"])
def test_first_call_of_a_process(program):
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.split() == ["0"], r.stdout + r.stderr
