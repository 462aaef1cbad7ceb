"""Low-rank adapters at widths that are whole blocks (K and N multiples of 64, R of 8 up to 64), whose operands go
through LDS."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import DEV, F32, rand  # noqa: E402
from test_gpu_lora import adapters  # noqa: E402

def test_refuses_y_in_part_of_its_operands():
    """Before anything is enqueued; views of one buffer that only touch are fine."""
    rng = np.random.default_rng(3)
    M, N, K, R = 4, 64, 128, 8
    buf = torch.zeros(4 * M * N, device=DEV)
    a = adapters(rng, 2, N, K, R)
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    base = buf[M * N:2 * M * N].view(M, N)
    base.copy_(rand(rng, (M, N), F32))
    x = buf[2 * M * N:2 * M * N + M * K].view(M, K)
    x.copy_(rand(rng, (M, K), F32))
    kept = buf.clone()
    for first in (1, M * N - 1, M * N + 1, 2 * M * N - 1, 2 * M * N, 2 * M * N + 7):
        with pytest.raises(tw.TwellError):
            tw.lora_add(x, a, index, base, y=buf[first:first + M * N].view(M, N))
    assert torch.equal(buf, kept)
    want = tw.lora_add(x, a, index, base)
    assert torch.equal(tw.lora_add(x, a, index, base, y=buf[:M * N].view(M, N)), want)
    assert torch.equal(tw.lora_add(x, a, index, base, y=base), want)
