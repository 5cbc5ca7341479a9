"""What the bounded waits inside the kernels left behind."""


def assert_none_gave_up(G, where: str) -> None:
    """Fails if a kernel's wait gave up since the last look, and clears the marks
    (the call itself returns GLU_OK: what it wrote is undefined then)."""
    words = {"block": G.block_device_errors(clear=True), "gated activation": G.glu_quant_device_errors(clear=True)}
    bad = {k: v for k, v in words.items() if any(v)}
    assert not bad, f"waits gave up in {where}: {bad}"
