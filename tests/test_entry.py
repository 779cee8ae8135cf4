"""The entry script: everything that it runs as a script is defined before it runs."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_script_runs_behind_its_definitions():
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    mains = [i for i, x in enumerate(body) if isinstance(x, ast.If)
             and any(isinstance(n, ast.Name) and n.id == "__name__" for n in ast.walk(x.test))]
    assert mains == [len(body) - 1]
