"""Every binding that takes ``stream=`` runs as a call on that stream, itself, with all of its arguments."""
import inspect

import pytest

from gated_deltanet_linear_eqs_b200 import api

CALLS = [f for n, f in vars(api).items() if n.startswith("gdn_") and "stream" in inspect.signature(f).parameters]


@pytest.mark.parametrize("f", CALLS, ids=lambda f: f.__name__)
def test_stream_argument(f, monkeypatch):
    seen = []
    monkeypatch.setattr(api, "_on", lambda stream, g, args: seen.append((stream, g, args)) or "called")
    names = [n for n in inspect.signature(f).parameters if n != "stream"]
    given = {n: object() for n in names}
    side = object()
    assert f(**given, stream=side) == "called"
    assert seen == [(side, f, {**given, "stream": side})]


def test_all_of_them():
    assert len(CALLS) == 29
