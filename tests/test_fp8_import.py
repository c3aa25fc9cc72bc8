"""The package on a torch that has no type for e8m0 scales: everything imports, and scales are torch.uint8."""
import subprocess
import sys


def test_imports_without_the_scales_type():
    code = ("import torch\n"
            "if hasattr(torch, 'float8_e8m0fnu'): del torch.float8_e8m0fnu\n"
            "import deepseek_v4_engram_gb300 as eg\n"
            "print(eg.engram_kv_append_fp8.__name__, eg.engram_attn_prompt.__name__)\n")
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
    assert done.stdout.split() == ["engram_kv_append_fp8", "engram_attn_prompt"]
