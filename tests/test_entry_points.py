"""The repository's entry points by their source: what they lean on."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_entry_point_brings_its_own_reference():
    """smoke() checks a block's operators without the helpers of their tests: it runs beside any tests folder that has
    the norm's tolerances and the step operators' forms."""
    tree = ast.parse(open(os.path.join(ROOT, "__graft_entry__.py")).read())
    used = set()
    for node in ast.walk(tree):
        if isinstance(node, ast.ImportFrom) and (node.module or "").split(".")[0] == "tests":
            used |= {n.name for n in node.names} if node.module == "tests" else {node.module.split(".")[1]}
        elif isinstance(node, ast.Import):
            used |= {n.name.split(".", 1)[1] for n in node.names if n.name.startswith("tests.")}
    assert used <= {"tolerances", "step_reference"}, used
