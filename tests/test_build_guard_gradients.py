"""The build rejects scratch memory in the gradients' products as well, whose waits are counted by hand too."""
import pytest

from moe_expert_dispatch_amd import build as b

_GRAD = "_ZN3moe12_GLOBAL__N_119grouped_grad_kernelILi3ENS0_5ShapeILi2ELi4ELi4ELi2ELi64EEELb1EEEvNS0_4ArgsE"


def _remarks(scratch, vspill):
    tag = "[-Rpass-analysis=kernel-resource-usage]"
    return "\n".join([f"x.hip:1:1: remark: Function Name: {_GRAD} {tag}",
                      f"x.hip:1:1: remark:     ScratchSize [bytes/lane]: {scratch} {tag}",
                      f"x.hip:1:1: remark:     VGPRs Spill: {vspill} {tag}"])


def test_scratch_in_a_gradient_is_rejected():
    b._check_no_scratch("gemm_grad.hip", _remarks(0, 0))
    for scratch, vspill in ((8, 0), (0, 2)):
        with pytest.raises(RuntimeError, match="grouped_grad_kernel"):
            b._check_no_scratch("gemm_grad.hip", _remarks(scratch, vspill))
