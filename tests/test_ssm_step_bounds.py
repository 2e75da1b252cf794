"""The bounds that the token step is held to see what they are for: x, B or C rounded to bf16 between the convolution and
the state update breaks them (planted in the fp64 form)."""
import pytest
import torch

import ssm_step_ref as step_ref

SHAPES = [(1, 2, 64, 1, 128), (3, 6, 16, 2, 16), (2, 3, 128, 1, 32), (5, 8, 64, 8, 64), (70, 4, 128, 2, 128),
          (1, 1, 16, 1, 128), (2, 2, 32, 2, 64)]


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,H,P,G,N", SHAPES, ids=str)
def test_rounding_between_the_parts_breaks_the_bounds(n, H, P, G, N, dtype, full):
    b = step_ref.inputs(n, H, P, G, N, dtype, seed=n + H)
    y, S, ty, tS, _ = step_ref.step(b, G, dtype, full)
    HP, GN = H * P, G * N
    for part, (first, last) in {"x": (0, HP), "B": (HP, HP + GN), "C": (HP + GN, HP + 2 * GN)}.items():
        def rounded(c):
            c = c.clone()
            c[:, first:last] = c[:, first:last].bfloat16().double()
            return c
        y2, S2 = step_ref.step(b, G, dtype, full, between=rounded)[:2]
        # x and B show in the state (in y they are weighed by steps of down to 1e-3), C in y where y itself is not bf16
        if part != "C":
            assert ((S2 - S).abs() > tS).double().mean() > 0.5, part
        elif dtype is torch.float32:
            assert ((y2 - y).abs() > ty).double().mean() > 0.5, part
