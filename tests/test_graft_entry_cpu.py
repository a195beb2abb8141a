"""The build and smoke entry points, run as a script (CPU)."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_script_part_comes_behind_every_function():
    """What `python __graft_entry__.py --smoke` calls is defined when it runs."""
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    script = [i for i, n in enumerate(body) if isinstance(n, ast.If)
              and any(isinstance(x, ast.Name) and x.id == "__name__" for x in ast.walk(n.test))]
    functions = {n.name: i for i, n in enumerate(body) if isinstance(n, ast.FunctionDef)}
    assert len(script) == 1 and script[0] > max(functions.values())
    called = {x.func.id for n in body for x in ast.walk(n) if isinstance(x, ast.Call) and isinstance(x.func, ast.Name)}
    assert {"build", "smoke", "smoke_serving"} <= called & set(functions)
