"""The host code of the gated product, the adapters and dropout under
AddressSanitizer, on the CPU, as test_abi_asan.py has the block's."""

import test_abi_operators_asan as operators


def test_mlp_host_code_under_address_sanitizer():
    operators.test_operators_host_code_under_address_sanitizer("test_abi_mlp.py")
