"""bench.py's --head-loss belongs to --prefetch: alone it is refused, not left out."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_head_loss_alone_is_refused(monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["bench.py", "--head-loss"])
    with pytest.raises(SystemExit) as stop:
        bench.parse()
    assert stop.value.code == 2
    assert "--head-loss goes with --prefetch" in capsys.readouterr().err


def test_head_loss_with_prefetch_is_taken(monkeypatch):
    monkeypatch.setattr(sys, "argv", ["bench.py", "--prefetch", "--head-loss"])
    args = bench.parse()
    assert args.prefetch and args.head_loss
