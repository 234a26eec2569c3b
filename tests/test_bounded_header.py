"""The public header declares every function that the library exports and the binding calls (no GPU)."""
import subprocess

import pytest

from transformer_decode_step_weight_gb300 import api, build


@pytest.fixture(scope="module")
def declared():
    build.build()
    return set(api.header_functions())


def test_exported_functions_are_declared(declared):
    out = subprocess.run(["nm", "-D", "--defined-only", api.LIB_PATH], capture_output=True, text=True, check=True).stdout
    names = {line.split()[-1] for line in out.splitlines()}
    exported = {n for n in names if n.startswith("qd_")}
    assert len(exported) >= 30 and not exported - declared


def test_bound_functions_are_declared(declared):
    assert not set(api._SIGS) - declared
