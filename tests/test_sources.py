"""Rules that every source of the library keeps, whatever it computes (no GPU needed)."""
import ast
import os
import textwrap

from mtp_speculative_draft_head_gb300 import build


def test_no_load_is_multicast():
    """Ranks of a replicated or sharded run load this one library: a copy that writes the shared memory of several
    CTAs at once stays out of all of it."""
    word = "multi" + "cast"
    for path in build._deps():
        with open(path) as f:
            assert word not in f.read(), os.path.basename(path)


def test_readme_step_decides_by_other_numbers_than_it_draws_with():
    """The documented speculative step: what `sample` draws with and what `verify` decides with are different arrays."""
    with open(os.path.join(build.ROOT, "README.md")) as f:
        text = f.read().split("A speculative step with sampled drafts:\n\n")[1]
    code = textwrap.dedent("\n".join(ln for ln in text.split("\n\n")[0].splitlines()))
    used = {}
    for call in (n for n in ast.walk(ast.parse(code)) if isinstance(n, ast.Call)):
        name = getattr(call.func, "attr", "")
        if name in ("sample", "verify"):
            arg = call.args[{"sample": 1, "verify": 3}[name]]
            used[name] = {n.id for n in ast.walk(arg) if isinstance(n, ast.Name)}
    assert used["sample"] and used["verify"] and not used["sample"] & used["verify"]
