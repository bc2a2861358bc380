"""What the first call on a device prepares: the state and the kernels that the
layer's calls share.  The kernels of the balance loss and of the 8-bit product are
prepared by their own calls, so that no other call loads them or fails for them.
CPU only (reads the sources)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_routed_expert_renorm_b200", "csrc")


def _read(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(code, head):
    """The braces after `head`."""
    i = code.index("{", code.index(head))
    depth = 0
    for j in range(i, len(code)):
        depth += {"{": 1, "}": -1}.get(code[j], 0)
        if depth == 0:
            return code[i:j + 1]
    raise AssertionError(head)


def test_shared_state_does_not_prepare_the_operators_kernels():
    body = _body(_read("coli_moe.cu"), "coli_status dev_info(DevInfo* out)")
    assert "ffn_splitk_kernel" in body
    assert "balance" not in body and "fp8" not in body


def test_each_operator_prepares_its_own():
    """Every entry point that launches kernels with more than the default shared
    memory asks for them; their launches sit in no other file."""
    ops = _read("ops_api.cuh")
    for entry, ready in (("coli_moe_balance(const float*", "balance"), ("coli_moe_balance_backward(", "balance"),
                         ("coli_fp8_matmul(", "fp8"), ("coli_moe_expert_ffn_fp8(", "fp8")):
        body = _body(ops, "coli_status " + entry)
        assert f"kernels_ready(di.dev, g_{ready}_ready, {ready}_kernels_ready)" in body, entry
    main = _read("coli_moe.cu")
    assert "launch_fp8" not in main and "launch_balance" not in main
