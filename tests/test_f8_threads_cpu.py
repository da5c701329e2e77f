"""First calls of the 8-bit family's tensor functions from several threads (no GPU).

A thread's first call fills the module's tables.  A trace stops it after each line of
that, and a call made then must find all the tables it uses or fill them itself."""
import sys

import pytest

from fp32_gemm_08_amd import f8

TABLES = ("_FORMAT_OF", "_TYPE_OF", "_F32", "_raw_stream", "_current_device")


@pytest.fixture
def fresh():
    held = {n: getattr(f8, n) for n in TABLES}
    for n in TABLES:
        setattr(f8, n, None)
    yield
    for n, v in held.items():
        setattr(f8, n, v)


def test_a_call_in_the_middle_of_anothers_first_one_finds_the_tables(fresh):
    torch = pytest.importorskip("torch")

    class OnGpu:
        device = torch.device("cuda", 0)

    seen = []

    def at_line(frame, event, arg):
        if event == "line":
            # what _device lets pass without filling the tables is complete
            seen.append(f8._FORMAT_OF is None or all(getattr(f8, n) is not None for n in TABLES))
        return at_line

    def at_call(frame, event, arg):
        return at_line if frame.f_code is f8._tables.__code__ else None

    before = sys.gettrace()
    sys.settrace(at_call)
    try:
        assert f8._device(OnGpu()) == OnGpu.device
    finally:
        sys.settrace(before)
    assert len(seen) >= 4 and all(seen)
    assert all(getattr(f8, n) is not None for n in TABLES)
