"""A test whose name a later one of its module takes never runs."""
import ast
import glob
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# the first of these runs as test_values_that_are_not_finite_of_every_type_and_through_each_activation
TWICE = {("test_gpu_dense.py", "test_values_that_are_not_finite_stay_in_their_rows_and_columns")}


def test_every_test_of_a_module_has_a_name_of_its_own():
    twice = set()
    for path in glob.glob(os.path.join(HERE, "test_*.py")):
        with open(path) as f:
            body = ast.parse(f.read()).body
        names = [n.name for n in body if isinstance(n, (ast.FunctionDef, ast.ClassDef))]
        twice |= {(os.path.basename(path), n) for n in names if names.count(n) > 1}
    assert twice == TWICE
