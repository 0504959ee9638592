"""The expert operators at the edges of what the header allows, against the 64-bit statements
(oracle/experts.py), with the tolerances of test_gpu_experts.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import experts as ex
from tests.test_gpu_experts import U, _close, _half_step, _np, _rand, _ws

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    return torch, nat


# ------------------------------------------------------------------ norm
def norm_grad_of(H, dtype, T=5):
    import torch

    from moe_expert_routing_top_gb300 import _native as nat
    s, w, dy = (_rand(torch, n, dtype, i) for i, n in enumerate(((T, H), (H,), (T, H))))
    rstd = torch.from_numpy(ex.rms_norm(_np(s), _np(w), 1e-6)[1]).float().cuda()
    dx, dw = torch.empty_like(s), torch.empty(H, device="cuda")
    n = nat.moer_rms_norm_workspace_bytes(T, H)
    nat.moer_rms_norm_grad(nat.make_norm(T=T, H=H, dtype=dtype, eps=1e-6, sum=s, weight=w, rstd=rstd, d_y=dy, d_x=dx, d_weight=dw), _ws(torch, n), n)
    rx, mx, rw, mw = ex.rms_norm_grad(_np(s), _np(w), _np(rstd), _np(dy))
    _close(dx, rx, (H + 24) * 2 * U * mx + _half_step(torch, dtype, rx), f"d_x of {H}")
    _close(dw, rw, (T + 16) * 2 * U * mw + 1e-44, f"d_weight of {H}")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_norm_gradient_next_to_48_KB(env, dtype):
    """Rows whose weight's gradient takes 48 KB of shared memory or a little less: with the kernel's own
    64 bytes they need more than a launch has by default.  In a process of its own, smallest first: a call with
    a longer row raises the kernel's limit for good."""
    code = f"from tests.test_gpu_expert_edges import norm_grad_of\nfor H in (12272, 12273, 12280, 12281, 12288, 12289, 12296): norm_grad_of(H, {dtype!r})"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
