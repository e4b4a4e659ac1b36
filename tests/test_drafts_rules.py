"""Rules that the drafted tokens' kernels keep, seen without a GPU: those that a run
cannot show, and the binding's."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_gqa_msa_gb300", "csrc")


def _code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_warp_group_moves_its_registers_in_one_place():
    """All warps of a warp group have to execute the same setmaxnreg: one call for the
    first group in front of the branch into its roles, one for the softmax groups."""
    code = _code("paged_tree.cu")
    assert len(re.findall(r"\bfewer_registers<k\w+>\(\)", code)) == 1
    assert len(re.findall(r"\bmore_registers<k\w+>\(\)", code)) == 1
    assert re.search(r"if \(warp < kSoftWarp0\) \{\s*fewer_registers<kOtherRegs>\(\);", code)
    # and that group is whole warp groups
    roles = dict(re.findall(r"\b(kCopyWarps|kCopyWarp0) = (\d+)", code))
    assert (int(roles["kCopyWarp0"]) + int(roles["kCopyWarps"])) % 4 == 0
