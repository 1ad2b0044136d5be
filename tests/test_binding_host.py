"""Host-side argument checks of the Python binding (no GPU): dtype, size and
device are checked before a pointer reaches the C library, which cannot check
them itself."""
import inspect
import os
import subprocess
import sys

import pytest
import torch

import speculative_decoding_verification_04_amd as sv


def test_arg_checks_dtype_size_and_device():
    t = torch.zeros(8, dtype=torch.int64)
    with pytest.raises(ValueError, match="must be int32"):
        sv._arg(t, "int32", 8, "draft")
    with pytest.raises(ValueError, match="needs at least 9 elements"):
        sv._arg(torch.zeros(8, dtype=torch.int32), "int32", 9, "draft")
    with pytest.raises(ValueError, match="must be on the GPU"):
        sv._arg(torch.zeros(8, dtype=torch.int32), "int32", 8, "draft")
    with pytest.raises(ValueError, match="is required"):
        sv._arg(None, "int32", 1, "draft")
    assert sv._arg(None, "int32", 1, "remaining", optional=True) is None
    with pytest.raises(ValueError, match="must be float64"):
        sv._arg(torch.zeros(4, dtype=torch.float32), "float64", 4, "final_mass", optional=True)


def test_unsupported_logit_dtype():
    with pytest.raises(ValueError, match="unsupported dtype"):
        sv._dtype_code(torch.zeros(2, dtype=torch.float16))


def test_the_package_and_its_build_import_without_torch():
    """Only calls need torch: the build module and the names are there without it."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "import speculative_decoding_verification_04_amd as sv\n"
            "from speculative_decoding_verification_04_amd import build\n"
            "print(sv.SPEC_ATTN_MAX_D, len(build.sources()) > 0, sv.SpecError.__name__)")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.split() == ["256", "True", "SpecError"], r.stderr


@pytest.mark.parametrize("call", ["mask", "rope", "rope_paged", "prompt", "prompt_paged", "tree", "tree_paged", "dtype"])
def test_any_call_may_be_the_first(call, monkeypatch):
    """No call reads a name that only an earlier call would have bound."""
    for name in ("torch", "_current_device", "_raw_stream"):
        monkeypatch.setattr(sv, name, None)
    kv, q, i = torch.zeros(1, 2, 2, 2, 8, 64), torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, dtype=torch.int32)
    run = {"mask": lambda: sv.spec_tree_mask(i, i, i, i, i),
           "rope": lambda: sv.spec_norm_rope_kv(q, q[:, :, :2], q[:, :, :2], kv, 0, i, i, q),
           "rope_paged": lambda: sv.spec_norm_rope_kv_paged(q, q[:, :, :2], q[:, :, :2], kv, 0, i, i, q),
           "prompt": lambda: sv.spec_prompt_attention(q[0], kv, 0, i, i, i, q[0]),
           "prompt_paged": lambda: sv.spec_prompt_attention_paged(q[0], kv, 0, i, i, i, q[0]),
           "tree": lambda: sv.spec_tree_attention(q, kv, 0, i, i, q, i),
           "tree_paged": lambda: sv.spec_tree_attention_paged(q, kv, 0, i, i, q, i),
           "dtype": lambda: sv._dtype_code(i)}[call]
    with pytest.raises(ValueError, match="must be on the GPU|unsupported dtype"):
        run()


@pytest.mark.parametrize("f", [sv.spec_tree_attention, sv.spec_tree_attention_paged])
def test_tree_attention_asks_for_its_workspace(f):
    """A default could only fail: the call cannot run without one."""
    assert inspect.signature(f).parameters["ws"].default is inspect.Parameter.empty
