"""The decode-step example runs: tokens chosen, rows forked, grown and dropped
and the cache packed, with every row's text as the host kept it."""

import pathlib
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = pathlib.Path(__file__).resolve().parents[1]


def test_decode_step_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from u32_prefix_scan_gb300 import build

    build.build()
    out = subprocess.run([sys.executable, str(ROOT / "examples" / "decode_step.py")], capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stderr
    assert "rows live on" in out.stdout
