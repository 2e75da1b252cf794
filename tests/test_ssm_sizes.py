"""Sizes beyond 2^31 - 1, which the C ABI's ints cannot say, are refused and not cut to 32 bits (no GPU; the tensors have
shapes only).  A token step of such a size has terabytes of state."""
import pytest
import torch

import gated_deltanet_linear_18_b200 as gdn

BIG = 2 ** 32 + 8


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_deltanet_linear_18_b200 import _build
    _build.build()


def t(*s, d=torch.bfloat16):
    return torch.empty(*s, dtype=d, device="meta")


def f(*s):
    return t(*s, d=torch.float32)


CU = t(2, d=torch.int32)
CALLS = {
    "conv rows": lambda: gdn.ssm_conv(t(1, BIG, 1), f(1, 4)),
    "conv channels": lambda: gdn.ssm_conv(t(1, 1, BIG), f(BIG, 4)),
    "packed conv rows": lambda: gdn.ssm_conv_varlen(t(BIG, 1), f(1, 4), None, CU, 8),
    "packed conv bound": lambda: gdn.ssm_conv_varlen(t(8, 1), f(1, 4), None, CU, 2 ** 32),
    "scan rows": lambda: gdn.ssm_scan(t(1, BIG, 1, 16), t(1, BIG, 1), f(1), t(1, BIG, 1, 16), t(1, BIG, 1, 16)),
    "packed scan rows": lambda: gdn.ssm_scan_varlen(t(BIG, 1, 16), t(BIG, 1), f(1), t(BIG, 1, 16), t(BIG, 1, 16), CU, 8),
    "packed scan bound": lambda: gdn.ssm_scan_varlen(t(8, 1, 16), t(8, 1), f(1), t(8, 1, 16), t(8, 1, 16), CU, 2 ** 32),
    "scan scratch": lambda: gdn.ssm_scan_workspace_bytes(3, 2 ** 32, 2, 1, 64, 64, torch.bfloat16),
    "packed scan scratch": lambda: gdn.ssm_scan_workspace_bytes(3, 8, 2, 1, 64, 64, torch.bfloat16, total=2 ** 32),
    "norm scratch": lambda: gdn.block_norm_bwd_workspace_bytes(4, BIG),
    "norm width": lambda: gdn.block_norm(t(1, BIG), t(1, BIG)),
    "norm backward width": lambda: gdn.block_norm_bwd(t(1, BIG), t(1, BIG), t(1, BIG)),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_refused(call):
    with pytest.raises(ValueError, match="below 2"):
        call()
