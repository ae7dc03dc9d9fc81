"""The operators around the attention in the bounds-checked debug build: their
own tests, in a child process that loads libveda_debug.so.  Each test there
that synchronises the library's status fails if a check fires."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_layer_operators_in_the_debug_build():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from tile_sparse_attention_head_b200 import build
    build.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_layer.py"), "-x", "-q", "-p",
                        "no:cacheprovider", "-k", "special or strides or block or chain or capture or gemm or norm_fp8"],
                       env=dict(os.environ, VEDA_DEBUG_BOUNDS="1"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


def test_rows_of_odd_shapes_in_the_debug_build():
    """The cases whose rows end inside a block or a group: the norm in both directions, the rotary operator, outputs at
    other borders and the calls under autograd."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from tile_sparse_attention_head_b200 import build
    build.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_layer.py"),
                        os.path.join(HERE, "test_gpu_layer_calls.py"), "-x", "-q", "-p", "no:cacheprovider", "-k",
                        "test_add_rms_norm or qkv_norm_rope or test_quant or calls or status or library"],
                       env=dict(os.environ, VEDA_DEBUG_BOUNDS="1"), capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
