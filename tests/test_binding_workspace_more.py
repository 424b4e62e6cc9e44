"""As test_binding_workspace: the workspace that the binding allocates lives until
the library function has returned, for the calls on pages, the verification of
drafted tokens and the adapters (stubs in place of the library and of tensors)."""
import pytest
import torch

from test_binding_workspace import Device, cache, stubbed  # noqa: F401

BF, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
d = Device

CALLS = {
    "kv4_reserve": lambda b: b.mxs_kv4_reserve(cache(b), d((2,), I32), d((3, 4), I32), d((3,), I32), d((4,), I32),
                                               slots=d((5,), I64), lens_out=d((3,), I32)),
    "verify_tree": lambda b: b.mxs_verify_tree(d((6, 100), BF), d((6,), I64), d((3,), I32), d((6,), F64),
                                               path=d((6,), I32), count=d((2,), I32), next_token=d((2,), I64)),
    "lora_add": lambda b: b.mxs_lora_add(d((6, 100), F32), d((6, 64), BF), d((6,), I32),
                                         b.LoraSet(d((4, 8, 64), BF), d((4, 100, 8), BF))),
}


@pytest.mark.parametrize("name", CALLS)
def test_workspace_of_the_binding_outlives_the_call(stubbed, name):  # noqa: F811
    binding, _ = stubbed
    CALLS[name](binding)
