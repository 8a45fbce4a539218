"""The example that runs scoring, distillation and adapters together."""
import pytest

from examples import recover_head
from tests.gpu_run import log

pytestmark = pytest.mark.gpu


def test_adapters_learn_two_teachers():
    r = recover_head.run(steps=30, hidden=256, vocab=3001, tokens=512, show=lambda s: log("[gpu] " + s))
    assert r["last"] < 0.5 * r["first"]
    assert r["with"] > r["without"] and r["agree_with"] > r["agree_without"]
    assert r["untouched"]
