"""examples/fp8_layer.py refuses counts below one by name (no GPU needed).  An empty prompt still took one token, for which the
pages were not counted."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("extra", [["--prompt", "0"], ["--steps", "0"], ["--batch", "0"], ["--prompt", "-3"]])
def test_counts_below_one(extra, monkeypatch, capsys):
    spec = importlib.util.spec_from_file_location("fp8_layer", os.path.join(ROOT, "examples", "fp8_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    monkeypatch.setattr("sys.argv", ["fp8_layer.py", *extra])
    with pytest.raises(SystemExit):
        module.main()
    assert "must be at least 1" in capsys.readouterr().err
