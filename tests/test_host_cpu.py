"""What the calls do on the host, without a GPU."""
import os

import pytest


@pytest.fixture(scope="module")
def lib():
    from dynamic_embedding_tables_amd import recis
    recis.load_library()
    return recis


def test_a_forked_process_asks_torch_before_it_launches(lib, monkeypatch):
    """torch refuses the GPU in a process that was forked off one that uses it: the handles kept to ask for the stream
    directly, which would not, are not a forked process's."""
    monkeypatch.setattr(lib, "_raw_stream", lambda device: 7 + device)
    monkeypatch.setattr(lib, "_current_device", lambda: 3)
    assert lib._stream() == 10
    pid = os.fork()
    if pid == 0:
        os._exit(0 if lib._raw_stream is None else 1)
    assert os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]) == 0
    assert lib._stream() == 10
