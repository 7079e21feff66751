"""Products on activations that the kernel right before them writes, which starts them
while it still runs: chains of calls on the same buffers, against the same calls one at
a time."""
import pytest
import torch

import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
N = 1024


def _weights(kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind in (dg.LINEAR_F16, dg.LINEAR_BF16):
        dt = torch.float16 if kind == dg.LINEAR_F16 else torch.bfloat16
        return {"W": (torch.randn(N, N, generator=g) * N ** -0.5).to(dt).to(DEV)}
    if kind == dg.LINEAR_W8A8:
        return {"W": torch.randint(-127, 128, (N, N), generator=g, dtype=torch.int8).to(DEV),
                "w_scale": torch.full((N,), 0.014 * N ** -0.5, device=DEV)}
    return {"W": torch.randint(0, 256, (N, N // 2), generator=g, dtype=torch.uint8).to(DEV),
            "w_scale": torch.full((N, N // 32), 0.21 * N ** -0.5, dtype=torch.float16, device=DEV)}


@pytest.mark.parametrize("M", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("kind", [dg.LINEAR_F16, dg.LINEAR_BF16, dg.LINEAR_W8A8, dg.LINEAR_W4A16, dg.LINEAR_W4A8])
def test_a_chain_of_calls_sees_the_call_before(kind, M):
    """norm -> (quantize) -> product -> residual add -> norm, 40 times over the same
    buffers with other inputs in each."""
    need_gpu()
    dt = torch.bfloat16 if kind == dg.LINEAR_BF16 else torch.float16
    steps = 40
    g = torch.Generator().manual_seed(5)
    starts = (torch.randn(steps, M, N, generator=g)).to(dt).to(DEV)
    h, x, y = (torch.zeros(M, N, dtype=dt, device=DEV) for _ in range(3))
    codes, scale = torch.zeros(M, N, dtype=torch.int8, device=DEV), torch.zeros(M, device=DEV)
    one = torch.ones(N, dtype=dt, device=DEV)
    w = _weights(kind, 6)
    a8 = kind in (dg.LINEAR_W8A8, dg.LINEAR_W4A8)
    op = dg.linear(kind, w["W"], M, N, N, w_scale=w.get("w_scale"), x=None if a8 else x, x_i8=codes if a8 else None,
                   x_scale=scale if a8 else None, y=y)
    ws = torch.zeros(max(dg.workspace_bytes([op]), 16), dtype=torch.uint8, device=DEV)

    def run(wait):
        outs = torch.zeros(steps, M, N, dtype=dt, device=DEV)
        pause = sync if wait else (lambda: None)
        for s in range(steps):
            calls = [lambda: dg.norm_residual(dg.norm(starts[s], h, x, one)),
                     (lambda: dg.quantize_act_i8(x, codes, scale)) if a8 else (lambda: None),
                     lambda: dg.linear_forward(op, ws),
                     lambda: dg.norm_residual(dg.norm(h, outs[s], x, one, y=y)),
                     (lambda: dg.quantize_act_i8(x, codes, scale)) if a8 else (lambda: None),
                     lambda: dg.linear_forward(op, ws),
                     lambda: dg.norm_residual(dg.norm(outs[s], None, outs[s], one, y=y))]
            for call in calls:
                call()
                pause()
        sync()
        return outs

    alone = run(True)
    assert torch.isfinite(alone.float()).all() and alone.float().std() > 0.5
    for _ in range(3):
        assert torch.equal(run(False), alone)
