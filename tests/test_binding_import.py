"""The binding's host-only calls need numpy and the library, not torch; the
calls that take tensors import it when they are made.  CPU only, each in a
process of its own."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HOST_CALLS = """
    from many_shot_icl_b200 import dbsa
    cfg = dbsa.DbsaConfig(8, 2, 128)
    offs = dbsa.group_blocks([5, 6, 7], 2)
    assert offs.tolist() == [0, 11, 18]
    assert dbsa.stage1_tile_count(cfg, offs) == len(dbsa.stage1_plan(cfg, offs)) > 0
    assert dbsa.encode_workspace_size(cfg, 18, 2) > 0
    assert dbsa.rope_tables_size(cfg, 100) > 0
    assert dbsa.shared_prefix_workspace_size(cfg, 3, 5, 100) > 0
"""


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from many_shot_icl_b200 import build
    build.build()


def run(code):
    p = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT,
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


def test_host_calls_without_torch():
    run("""
    import sys
    sys.modules["torch"] = None      # importing it raises ImportError
    """ + HOST_CALLS)


def test_host_calls_do_not_import_torch():
    run("    import sys" + HOST_CALLS + """
    assert "torch" not in sys.modules
    """)


def test_a_torch_without_cuda_names():
    """A build of torch for the CPU: host calls work, and calls that take tensors
    refuse CPU tensors as they do with any build."""
    run("""
    import torch
    del torch._C._cuda_getCurrentRawStream
    """ + HOST_CALLS + """
    i32 = dict(dtype=torch.int32)
    pages = torch.zeros(4, 2, 64, 128, dtype=torch.bfloat16)
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    try:
        dbsa.paged_append(cfg, rows, rows, pages, pages, torch.zeros(3, 1, **i32),
                          torch.zeros(4, **i32), torch.zeros(3, **i32),
                          torch.zeros(1 << 16, dtype=torch.uint8))
    except dbsa.DbsaError as e:
        assert e.status == dbsa.ERR_INVALID_ARG and "CUDA device" in str(e)
    else:
        raise AssertionError("not refused")
    """)
