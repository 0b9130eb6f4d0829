"""The serving example with its pool, block scales and drafts."""
import os
import re
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("more", [["--blocks"], ["--drafts", "3"], ["--e4m3", "--drafts", "2"],
                                  ["--blocks", "--drafts", "4"]])
def test_example_with_drafts(more, capsys, monkeypatch):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import serve_block
    finally:
        sys.path.pop(0)
    monkeypatch.setattr(sys, "argv", ["serve_block.py", "--experts", "4", "--seqs", "3", "--prompt", "150",
                                      "--chunk", "64", "--steps", "5", *more])
    serve_block.main()
    text = capsys.readouterr().out
    assert "lengths now [156, 119, 82]" in text and "device status 0" in text
    if "--drafts" in more:
        # every step of the 1 + 5 keeps a token at least and its drafts at most
        after = [int(x) for x in re.findall(r"lengths now \[([^]]*)\]", text)[1].split(", ")]
        most = int(more[more.index("--drafts") + 1]) + 1
        for a, b in zip([156, 119, 82], after):
            assert a + 6 <= b <= a + 6 * most
