"""Host-only checks of the speculative-decoding operators at the edges of what their
documentation allows."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_fp8_b200", "csrc")


def _code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_tree_attention_has_no_unbounded_wait_in_its_roles():
    """After a wait that ran out, warps leave their loops one by one, so nothing inside them may wait for a number
    of threads: a named barrier there could wait for warps that have left, for ever.  (Named barriers
    would be the only such wait besides __syncthreads, which stands before and behind the loops.)"""
    code = _code("tree_attn.cu")
    assert not re.search(r"\bbar(rier)?(\.cta)?\.(sync|red|arrive)\b", code)
    body = code[code.index("void tree_attn_body("):code.index("void __launch_bounds__(TA_THREADS")]
    roles = body[body.index("if (warp < 4 || warp >= 12)"):body.rindex("if (ctl->abort)")]
    assert roles.count("__syncthreads") == 1 and roles.rindex("__syncthreads") > roles.rindex("mbar_arrive(&oempty")
    assert "mbar_wait(" not in roles and "mbar_try_wait(" not in roles
